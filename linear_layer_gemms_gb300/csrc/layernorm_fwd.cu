// LayerNorm forward (include/layernorm_forward.h): per row mean, variance, rstd, and
// out = (x - mean) * rstd * weight + bias.
//
// Bound by HBM: each row read once and written once. A team of P warps owns a
// row and keeps it in registers (VPT 16-byte vectors per thread), so the
// variance is the mean of the squared differences, formed after the mean
// without a second read, and no cancellation is paid for it. Sums: in the
// thread, an xor butterfly over the warp, the warps in order. Rows wider than
// the largest team holds are read three times (mean, variance, output), the
// second and third time from L2.
#include "../../include/layernorm_forward.h"
#include "ops.h"
#include "ptx.cuh"
#include "q8.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

namespace mmbwd {
namespace {

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    // value e of a vector, plus c
    __device__ static float plus(const uint4& v, int e, float c) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        return __uint_as_float(w[e]) + c;
    }
    __device__ static void get(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static float plus(const uint4& v, int e, float c) {  // one instruction, without unpacking
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float r;
        if (e & 1)
            asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, b, %2;}" : "=f"(r) : "r"(w[e >> 1]), "f"(c));
        else
            asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, a, %2;}" : "=f"(r) : "r"(w[e >> 1]), "f"(c));
        return r;
    }
    __device__ static void get(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 put(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The sum of the team's P warp sums, in warp order, in every thread. `slot`:
// 2 P floats of the team's; `which` alternates, so that one barrier per sum is enough.
template <int P>
__device__ __forceinline__ float team_sum(float s, float* slot, int which, int warp_in_team, int team) {
    s = warp_sum(s);
    if constexpr (P == 1) {
        return s;
    } else {
        float* at = slot + which * P;
        if ((threadIdx.x & 31) == 0) at[warp_in_team] = s;
        ptx::named_bar_sync(static_cast<uint32_t>(1 + team), 32 * P);
        float t = at[0];
#pragma unroll
        for (int w = 1; w < P; ++w) t += at[w];
        return t;
    }
}

// A row's mean from its sum. The product with the rounded 1 / C alone can miss the
// quotient by a step, and a constant row would not give the bias; one correction by
// the remainder, which a fused multiply-add forms exactly, makes the mean of an exact
// sum exact: the remainder is (mean - q) C, and its product with 1 / C is mean - q to
// one part in 2^23, far below the half step at which q + (mean - q) rounds to the mean.
// (Quotients in their place: 8192 x 768 bf16 4.3 -> 4.8 us from L2, this: 4.3.) An
// infinite sum has no remainder and stays as it is.
__device__ __forceinline__ float mean_of(float sum, int C, float inv_c) {
    const float q = sum * inv_c, rest = fmaf(-q, static_cast<float>(C), sum);
    return rest == rest ? fmaf(rest, inv_c, q) : q;
}

// Teams of one warp share a block of four rows; larger teams are a block.
template <int P>
constexpr int TEAMS_PER_BLOCK = P == 1 ? 4 : 1;

// AHEAD: the blocks are as many as are resident and each thread has its next
// row's vectors in flight while it works on one; otherwise a team per row.
template <typename T, int P, int VPT, bool AHEAD>
__global__ void __launch_bounds__(32 * P * TEAMS_PER_BLOCK<P>)
    ln_fwd_kernel(T* out, float* mean_out, float* rstd_out, const T* inp, const T* __restrict__ weight,
                  const T* __restrict__ bias, int64_t rows, int C, float inv_c, float eps) {
    using V = Vec<T>;
    constexpr int N = V::N;
    constexpr int TEAMS = TEAMS_PER_BLOCK<P>;
    __shared__ float slots[TEAMS][2 * P];
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int team = warp / P, wt = warp % P, t = wt * 32 + lane;
    const int nvec = C / N;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    // A row's vectors as they are stored: 16 bytes of registers each, so that the
    // next row fits beside it; the differences from the mean are formed twice.
    uint4 x[VPT], next[VPT];
    auto fetch = [&](uint4 (&to)[VPT], int64_t r) {
        const uint4* xr = reinterpret_cast<const uint4*>(inp + r * C);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = t + 32 * P * j;
            to[j] = j + 1 < VPT || v < nvec ? xr[v] : make_uint4(0u, 0u, 0u, 0u);  // only the last vector may be missing
        }
    };
    int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
    if (r < rows) fetch(x, r);
    for (; r < rows; r += stride) {
        if (AHEAD && r + stride < rows) fetch(next, r + stride);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) s = V::plus(x[j], e, s);
        const float mean = mean_of(team_sum<P>(s, slots[team], 0, wt, team), C, inv_c);
        s = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const bool on = j + 1 < VPT || t + 32 * P * j < nvec;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = on ? V::plus(x[j], e, -mean) : 0.f;
                s += d * d;
            }
        }
        const float var = team_sum<P>(s, slots[team], 1, wt, team) * inv_c;
        const float rstd = 1.f / sqrtf(var + eps);
        uint4* dst = reinterpret_cast<uint4*>(out + r * C);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = t + 32 * P * j;
            if (j + 1 < VPT || v < nvec) {
                float y[N], w[N], b[N];
                V::get(__ldg(reinterpret_cast<const uint4*>(weight) + v), w);
                V::get(bias ? __ldg(reinterpret_cast<const uint4*>(bias) + v) : make_uint4(0u, 0u, 0u, 0u), b);
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = V::plus(x[j], e, -mean) * rstd * w[e] + b[e];
                __stcs(dst + v, V::put(y));
            }
            if (AHEAD) x[j] = next[j];
        }
        if (t == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        if (!AHEAD) break;
    }
}

// Rows wider than a team of 32 warps holds: a block of 32 warps per row, read
// three times, four vectors a thread in flight (100 x 131072 bf16 16.1 us; two: 25.3).
template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(T* out, float* mean_out, float* rstd_out, const T* inp,
                                                           const T* __restrict__ weight, const T* __restrict__ bias,
                                                           int64_t rows, int C, float inv_c, float eps) {
    using V = Vec<T>;
    constexpr int N = V::N;
    __shared__ float slots[2 * 32];
    const int t = static_cast<int>(threadIdx.x), wt = t >> 5;
    const int nvec = C / N;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const uint4* xr = reinterpret_cast<const uint4*>(inp + r * C);
        float s = 0.f;
#pragma unroll 4
        for (int v = t; v < nvec; v += 1024) {
            float f[N];
            V::get(xr[v], f);
#pragma unroll
            for (int e = 0; e < N; ++e) s += f[e];
        }
        const float mean = mean_of(team_sum<32>(s, slots, 0, wt, 0), C, inv_c);
        s = 0.f;
#pragma unroll 4
        for (int v = t; v < nvec; v += 1024) {
            float f[N];
            V::get(xr[v], f);
#pragma unroll
            for (int e = 0; e < N; ++e) s += (f[e] - mean) * (f[e] - mean);
        }
        const float var = team_sum<32>(s, slots, 1, wt, 0) * inv_c;
        const float rstd = 1.f / sqrtf(var + eps);
#pragma unroll 4
        for (int v = t; v < nvec; v += 1024) {
            float f[N], w[N], b[N];
            V::get(xr[v], f);
            V::get(__ldg(reinterpret_cast<const uint4*>(weight) + v), w);
            V::get(bias ? __ldg(reinterpret_cast<const uint4*>(bias) + v) : make_uint4(0u, 0u, 0u, 0u), b);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = (f[e] - mean) * rstd * w[e] + b[e];
            reinterpret_cast<uint4*>(out + r * C)[v] = V::put(f);
        }
        if (t == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
    }
}

template <typename T>
using LnFwdKernel = void (*)(T*, float*, float*, const T*, const T*, const T*, int64_t, int, float, float);

template <typename T>
struct Choice {
    LnFwdKernel<T> kernel;
    int threads;
    bool ahead;
};

// The kernel whose team of P warps holds a row in exactly `need` vectors a
// thread, VPT at least and eight at most.
template <typename T, int P, int VPT, bool AHEAD>
Choice<T> pick(int need) {
    if constexpr (VPT < 8) {
        if (need > VPT) return pick<T, P, VPT + 1, AHEAD>(need);
    }
    return {ln_fwd_kernel<T, P, VPT, AHEAD>, 32 * P * TEAMS_PER_BLOCK<P>, AHEAD};
}

// By the row's 16-byte vectors: a warp per row up to eight vectors a lane (no
// barrier), then teams that fill most of their lanes. The next row is fetched ahead
// where its registers fit beside the current row's. Measured (us), AHEAD / not:
// 8192 x 1600 bf16 (one warp) 10.5 / 11.4; 4000 x 2400 bf16 (4 warps, 3 vectors) 8.4 /
// 9.5, with 8 warps 12.5; with two warps a row 8192 x 1600 takes 11.3; 2000 x 6400 bf16 (4 warps, 7) 10.6 / 12.8, fp32 8192 x 3200
// 34.9 / 32.4; 4096 x 8192 fp32 (8 warps, 8) 46.7 / 41.4.
template <typename T>
Choice<T> choose(int nvec) {
    if (nvec <= 32 * 8) return pick<T, 1, 1, true>((nvec + 31) / 32);
    if (nvec <= 128 * 4) return pick<T, 4, 3, true>((nvec + 127) / 128);
    if (nvec <= 128 * 8) return pick<T, 4, 5, sizeof(T) == 2>((nvec + 127) / 128);
    if (nvec <= 256 * 8) return pick<T, 8, 5, false>((nvec + 255) / 256);
    if (nvec <= 512 * 8) return pick<T, 16, 5, false>((nvec + 511) / 512);
    if (nvec <= 1024 * 8) return pick<T, 32, 5, false>((nvec + 1023) / 1024);
    return {ln_fwd_wide_kernel<T>, 1024, true};
}

template <typename T>
cudaError_t launch(T* out, float* mean, float* rstd, const T* inp, const T* weight, const T* bias, int64_t BT, int C,
                   float eps, int num_sms, cudaStream_t stream) {
    const Choice<T> c = choose<T>(C / Vec<T>::N);
    const int teams = C / Vec<T>::N <= 32 * 8 ? TEAMS_PER_BLOCK<1> : 1;
    int64_t blocks = (BT + teams - 1) / teams;
    if (c.ahead) {
        int per_sm = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, c.kernel, c.threads, 0);
        if (e != cudaSuccess) return e;
        blocks = std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * std::max(per_sm, 1));
    }
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(c.threads), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float inv_c = 1.f / static_cast<float>(C);
    return cudaLaunchKernelEx(&cfg, c.kernel, out, mean, rstd, inp, weight, bias, BT, C, inv_c, eps);
}

}  // namespace

cudaError_t ln_forward_launch(void* out, float* mean, float* rstd, const void* inp, const void* weight,
                              const void* bias, int64_t BT, int C, float eps, int dtype, int num_sms,
                              cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    if (dtype == MMBWD_F32)
        return launch(static_cast<float*>(out), mean, rstd, static_cast<const float*>(inp),
                      static_cast<const float*>(weight), static_cast<const float*>(bias), BT, C, eps, num_sms, stream);
    return launch(static_cast<__nv_bfloat16*>(out), mean, rstd, static_cast<const __nv_bfloat16*>(inp),
                  static_cast<const __nv_bfloat16*>(weight), static_cast<const __nv_bfloat16*>(bias), BT, C, eps,
                  num_sms, stream);
}

}  // namespace mmbwd
