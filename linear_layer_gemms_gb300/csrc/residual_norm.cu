// The step between two blocks (include/residual_norm.h): residual_out = x + scale * gate *
// post(branch), out = norm(residual_out), and its gradients.
//
// Bound by HBM. Forward: two rows read, two written. A team of P warps owns a row and
// keeps it in registers (VPT 16-byte vectors per thread) from the branch's statistics to
// the output, so nothing is read twice and each variance comes from the differences
// (LAYER) of values at hand. Backward: four rows read, two written. A team owns a row as
// well, a thread 8 or 16 columns of it; it has the next rows in flight, forms the row's
// four sums in two rounds and keeps its columns' parameter sums in registers over all
// rows of the team. Rows that no team holds (C > 8192 in bf16, 6144 in fp32) take two
// passes: one forms the rows' sums, one goes down column tiles.
#include "../../include/residual_norm.h"
#include "ops.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

namespace mmbwd {
namespace {

constexpr int NONE = LNBWD_NORM_NONE, LAYER = LNBWD_NORM_LAYER;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void get(const uint4& v, float* f) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 put(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void get(const uint4& v, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 put(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The values of vector v of a tensor that may be absent (then `fill`).
template <typename T>
__device__ __forceinline__ void column(const void* p, int v, float fill, float (&f)[Vec<T>::N]) {
    if (p) {
        Vec<T>::get(__ldg(reinterpret_cast<const uint4*>(p) + v), f);
    } else {
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) f[e] = fill;
    }
}

// Two fp32 values side by side: one instruction works on both, so these kernels issue
// fewer (8.0 million instead of 13.5 for 8192 x 1600).
struct F2 {
    unsigned long long v;
    __device__ static F2 of(float a, float b) {
        F2 r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
        return r;
    }
    __device__ static F2 both(float a) { return of(a, a); }
    __device__ float lo() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ float hi() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// A 16-byte vector as pairs of fp32 values, and back.
template <typename T>
struct Pairs;
template <>
struct Pairs<float> {
    static constexpr int H = 2;
    __device__ static void get(const uint4& v, F2* f) {
        f[0] = F2::of(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = F2::of(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static uint4 put(const F2* f) {
        return make_uint4(__float_as_uint(f[0].lo()), __float_as_uint(f[0].hi()), __float_as_uint(f[1].lo()), __float_as_uint(f[1].hi()));
    }
};
template <>
struct Pairs<__nv_bfloat16> {
    static constexpr int H = 4;
    __device__ static void get(const uint4& v, F2* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = F2::of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ static uint4 put(const F2* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].lo(), f[i].hi());
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

// The sums of R values over a team's P warps, in warp order, in every thread. Consecutive
// sums alternate between two sets of slots, so that one barrier per sum is enough.
template <int P, int R>
struct TeamSum {
    float* slots;  // 2 P R floats
    int warp, team, which = 0;
    __device__ void operator()(float (&s)[R]) {
#pragma unroll
        for (int k = 0; k < R; ++k) s[k] = warp_sum(s[k]);
        if constexpr (P > 1) {
            float* at = slots + which * (P * R);
            which ^= 1;
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int k = 0; k < R; ++k) at[warp * R + k] = s[k];
            }
            ptx::named_bar_sync(static_cast<uint32_t>(1 + team), 32 * P);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                s[k] = at[k];
#pragma unroll
                for (int w = 1; w < P; ++w) s[k] += at[w * R + k];
            }
        }
    }
};

// A row's mean from its sum: the product with the rounded 1 / C, corrected by its
// remainder, so that the mean of an exact sum is exact and a row of one value has no
// differences from it. An infinite sum has no remainder and stays as it is.
__device__ __forceinline__ float mean_of(float sum, int C, float inv_c) {
    const float q = sum * inv_c, rest = fmaf(-q, static_cast<float>(C), sum);
    return rest == rest ? fmaf(rest, inv_c, q) : q;
}

// Teams of a block: four warps' worth, one team of more.
template <int P>
constexpr int TEAMS = P < 4 ? 4 / P : 1;

struct Forward {
    ResidualNorm a;
    float inv_c;
};

// Mean (0 without one) and rstd of the team's R rows v; the values beyond a row are zero
// and `last` says whether the last vector is in it.
template <int P, int R, int VPT, int H>
__device__ __forceinline__ void statistics(const F2 (&v)[R][VPT * H], bool layer, bool last, int C, float inv_c, float eps,
                                           TeamSum<P, R>& sum, float (&mean)[R], float (&rstd)[R]) {
    float s[R];
#pragma unroll
    for (int k = 0; k < R; ++k) mean[k] = 0.f;
    if (layer) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            F2 t = v[k][0];
#pragma unroll
            for (int i = 1; i < VPT * H; ++i) t = add2(t, v[k][i]);
            s[k] = t.lo() + t.hi();
        }
        sum(s);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] = mean_of(s[k], C, inv_c);
            const F2 m = F2::both(-mean[k]);
            F2 t = F2::both(0.f), u = F2::both(0.f);  // u: the last vector's
#pragma unroll
            for (int i = 0; i < VPT * H; ++i) {
                const F2 d = add2(v[k][i], m);
                if (i < (VPT - 1) * H) t = fma2(d, d, t);
                else u = fma2(d, d, u);
            }
            s[k] = t.lo() + t.hi() + (last ? u.lo() + u.hi() : 0.f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            F2 t = F2::both(0.f);
#pragma unroll
            for (int i = 0; i < VPT * H; ++i) t = fma2(v[k][i], v[k][i], t);
            s[k] = t.lo() + t.hi();
        }
    }
    sum(s);
#pragma unroll
    for (int k = 0; k < R; ++k) rstd[k] = 1.f / sqrtf(fmaf(s[k], inv_c, eps));
}

// 16 bytes on their way from global into shared memory.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait_but() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// R rows at a time to a team: the columns' weights are read and unpacked once for all of
// them. AHEAD: the blocks are as many as are resident, and while a team works on its rows
// the next ones are on their way into shared memory, each thread's vectors to places that
// only it reads (no barrier); otherwise every team has R rows, loaded into registers.
template <typename T, int P, int VPT, int R, bool AHEAD>
__global__ void __launch_bounds__(32 * P * TEAMS<P>) residual_forward_kernel(const __grid_constant__ Forward f) {
    constexpr int N = Vec<T>::N, H = Pairs<T>::H, THREADS = 32 * P * TEAMS<P>;
    extern __shared__ __align__(16) uint8_t buffer[];
    __shared__ float slots[TEAMS<P>][2 * P * R];
    const ResidualNorm& a = f.a;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int team = warp / P, wt = warp % P, t = wt * 32 + lane;
    const int nvec = a.C / N;
    const bool last = t + 32 * P * (VPT - 1) < nvec;
    const uint32_t mine = ptx::smem_u32(buffer) + threadIdx.x * 16u;  // vector j of row k: at (k VPT + j) * 16 * THREADS
    constexpr uint32_t X = R * VPT * THREADS * 16u;                   // the branch's vectors, then x's
    if (AHEAD && !last) {  // what is beyond a row stays zero
#pragma unroll
        for (int k = 0; k < R; ++k) {
            ptx::sts128u(mine + (k * VPT + VPT - 1) * (THREADS * 16), make_uint4(0u, 0u, 0u, 0u));
            ptx::sts128u(mine + X + (k * VPT + VPT - 1) * (THREADS * 16), make_uint4(0u, 0u, 0u, 0u));
        }
    }
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS<P> * R;
    auto request = [&](const void* p, uint32_t to, int64_t r0) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r0 + k < a.rows) {
                const uint4* row = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + (r0 + k) * a.C);
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (j + 1 < VPT || last) copy16(to + (k * VPT + j) * (THREADS * 16), row + t + 32 * P * j);
            }
        }
        copies_commit();
    };
    TeamSum<P, R> sum{slots[team], wt, team};
    // The weights of a thread's columns as they are stored, requested ahead of the sums that
    // they are needed behind (loaded where they are used, 8192 x 1600 with two LayerNorms
    // took 36 us instead of 25); kept over all rows where a thread has few columns.
    constexpr bool KEEP = AHEAD && VPT <= 2;
    static_assert(R == 1 || AHEAD, "rows that are loaded come one at a time");
    constexpr bool LATE = !AHEAD && VPT > 1;  // 64 registers: x and the weights are fetched where they are used
    uint4 gate[VPT], weight_post[VPT], bias_post[VPT], weight[VPT], bias[VPT];
    auto column_of = [&](const void* p, int j) {
        return p && (j + 1 < VPT || last) ? __ldg(static_cast<const uint4*>(p) + t + 32 * P * j) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto columns = [&](const void* p, uint4 (&to)[VPT]) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) to[j] = column_of(p, j);
    };
    if (KEEP) {
        columns(a.gate, gate);
        columns(a.weight_post, weight_post);
        columns(a.bias_post, bias_post);
        columns(a.weight, weight);
        columns(a.bias, bias);
    }
    int64_t r0 = (static_cast<int64_t>(blockIdx.x) * TEAMS<P> + team) * R;
    if (AHEAD) {
        request(a.branch, mine, r0);
        request(a.x, mine + X, r0);
    }
    for (; r0 < a.rows; r0 += step) {
        bool there[R];  // (nothing is stored of a row that is not)
#pragma unroll
        for (int k = 0; k < R; ++k) there[k] = r0 + k < a.rows;
        uint4 x[R][VPT];
        F2 v[R][VPT * H];
        if constexpr (AHEAD) {
            copies_wait_but<1>();  // (x's request is the younger one)
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < VPT; ++j) Pairs<T>::get(ptx::lds128(mine + (k * VPT + j) * (THREADS * 16)), v[k] + j * H);
            request(a.branch, mine, r0 + step);
        } else {
            auto load = [&](const void* p, int k, int j) {
                return (j + 1 < VPT || last) && there[k]
                           ? reinterpret_cast<const uint4*>(static_cast<const T*>(p) + (r0 + k) * a.C)[t + 32 * P * j]
                           : make_uint4(0u, 0u, 0u, 0u);
            };
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    if (!LATE) x[k][j] = load(a.x, k, j);
                    Pairs<T>::get(load(a.branch, k, j), v[k] + j * H);
                }
        }
        float mean[R], rstd[R];
        if (!KEEP && !LATE) {
            columns(a.gate, gate);
            columns(a.weight_post, weight_post);
            columns(a.bias_post, bias_post);
        }
        if (a.post != NONE) {
            statistics<P, R, VPT, H>(v, a.post == LAYER, last, a.C, f.inv_c, a.eps, sum, mean, rstd);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (t == 0 && there[k] && a.mean_post) a.mean_post[r0 + k] = mean[k];
                if (t == 0 && there[k] && a.rstd_post) a.rstd_post[r0 + k] = rstd[k];
            }
        }
        if constexpr (AHEAD) {
            copies_wait_but<1>();  // (the next branch's is the younger one)
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < VPT; ++j) x[k][j] = ptx::lds128(mine + X + (k * VPT + j) * (THREADS * 16));
            request(a.x, mine + X, r0 + step);
        }
        auto out_row = [&](void* p, int k) { return reinterpret_cast<uint4*>(static_cast<T*>(p) + (r0 + k) * a.C); };
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = t + 32 * P * j;
            if (j + 1 < VPT || last) {
                if (LATE) gate[j] = column_of(a.gate, j), weight_post[j] = column_of(a.weight_post, j), bias_post[j] = column_of(a.bias_post, j);
                F2 up[H];  // scale * gate
                if (a.gate) {
                    Pairs<T>::get(gate[j], up);
#pragma unroll
                    for (int i = 0; i < H; ++i) up[i] = mul2(up[i], F2::both(a.scale));
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) up[i] = F2::both(a.scale);
                }
                if (a.post != NONE) {
                    F2 w[H];
                    Pairs<T>::get(weight_post[j], w);
                    if (a.post == LAYER) {
                        F2 b[H];
                        Pairs<T>::get(bias_post[j], b);
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int i = 0; i < H; ++i)
                                v[k][j * H + i] = fma2(mul2(add2(v[k][j * H + i], F2::both(-mean[k])), F2::both(rstd[k])), w[i], b[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < H; ++i) up[i] = mul2(up[i], w[i]);
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int i = 0; i < H; ++i) v[k][j * H + i] = mul2(v[k][j * H + i], F2::both(rstd[k]));
                    }
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    F2 xv[H];
                    if constexpr (LATE) x[k][j] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + r0 * a.C)[c];
                    Pairs<T>::get(x[k][j], xv);
#pragma unroll
                    for (int i = 0; i < H; ++i) v[k][j * H + i] = fma2(up[i], v[k][j * H + i], xv[i]);
                    if (there[k]) out_row(a.residual_out, k)[c] = Pairs<T>::put(v[k] + j * H);
                }
            }
        }
        if (a.norm != NONE) {
            if (!KEEP && !LATE) {
                columns(a.weight, weight);
                columns(a.bias, bias);
            }
            statistics<P, R, VPT, H>(v, a.norm == LAYER, last, a.C, f.inv_c, a.eps, sum, mean, rstd);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (t == 0 && there[k] && a.mean) a.mean[r0 + k] = mean[k];
                if (t == 0 && there[k] && a.rstd) a.rstd[r0 + k] = rstd[k];
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = t + 32 * P * j;
                if (j + 1 < VPT || last) {
                    if (LATE) weight[j] = column_of(a.weight, j), bias[j] = column_of(a.bias, j);
                    F2 w[H];
                    Pairs<T>::get(weight[j], w);
                    if (a.norm == LAYER) {
                        F2 b[H];
                        Pairs<T>::get(bias[j], b);
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int i = 0; i < H; ++i)
                                v[k][j * H + i] = fma2(mul2(add2(v[k][j * H + i], F2::both(-mean[k])), F2::both(rstd[k])), w[i], b[i]);
                    } else {
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int i = 0; i < H; ++i) v[k][j * H + i] = mul2(mul2(v[k][j * H + i], F2::both(rstd[k])), w[i]);
                    }
#pragma unroll
                    for (int k = 0; k < R; ++k)
                        if (there[k]) __stcs(out_row(a.out, k) + c, Pairs<T>::put(v[k] + j * H));
                }
            }
        }
        if (!AHEAD) break;
    }
}

// Dynamic shared memory of a kernel allowed up to `bytes` on the current device, once; the
// caller holds the library's lock.
template <auto kernel>
cudaError_t allow_smem(int bytes) {
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <typename T, int P, int VPT, int R, bool AHEAD>
cudaError_t launch_forward(const Forward& f, int num_sms, cudaStream_t stream) {
    constexpr auto kernel = residual_forward_kernel<T, P, VPT, R, AHEAD>;
    constexpr int threads = 32 * P * TEAMS<P>, smem = AHEAD ? 2 * R * VPT * threads * 16 : 0;
    int64_t blocks = (f.a.rows + TEAMS<P> * R - 1) / (TEAMS<P> * R);
    if (AHEAD) {
        int per_sm = 0;
        cudaError_t e = allow_smem<kernel>(smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        blocks = std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * std::max(per_sm, 1));
    }
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, f);
}

// The kernel whose team holds a row in exactly `need` vectors a thread, VPT to MOST.
template <typename T, int P, int VPT, int MOST, int R, bool AHEAD>
cudaError_t launch_team(const Forward& f, int need, int num_sms, cudaStream_t stream) {
    if constexpr (VPT < MOST) {
        if (need > VPT) return launch_team<T, P, VPT + 1, MOST, R, AHEAD>(f, need, num_sms, stream);
    }
    return launch_forward<T, P, VPT, R, AHEAD>(f, num_sms, stream);
}

// By the row's 16-byte vectors. Measured, us (post and norm RMS with a gate / norm LAYER
// alone, bf16): 8192 x 768 a warp per row 11.1 / 10.4, four warps and two rows 11.8 / 11.4;
// 8192 x 1600 four warps and two rows at a time 19.8 / 19.5, a warp 21.6 / 20.2, two warps 21.9
// / 20.7, eight 24.2 / 22.6; 4096 x 4096 eight warps 24.3 / 24.1, with two rows 27.2 / 26.1, sixteen 29.1
// / 27.4; 2000 x 8192 eight warps of four vectors 24.2 / 23.0, sixteen of two 25.0 / 24.8. Few
// rows: as many warps as have a vector each, one row (512 x 1600 3.4, 1 x 1600 2.1; in teams
// of two warps 4.7 and 3.3).
template <typename T>
cudaError_t forward(const ResidualNorm& a, int num_sms, cudaStream_t stream) {
    const Forward f{a, 1.f / static_cast<float>(a.C)};
    const int nvec = a.C / Vec<T>::N;
    if (a.rows <= 4 * num_sms && nvec <= 1024) {
        if (nvec <= 32) return launch_forward<T, 1, 1, 1, false>(f, num_sms, stream);
        if (nvec <= 64) return launch_forward<T, 2, 1, 1, false>(f, num_sms, stream);
        if (nvec <= 128) return launch_forward<T, 4, 1, 1, false>(f, num_sms, stream);
        if (nvec <= 256) return launch_forward<T, 8, 1, 1, false>(f, num_sms, stream);
        if (nvec <= 512) return launch_forward<T, 16, 1, 1, false>(f, num_sms, stream);
        return launch_forward<T, 32, 1, 1, false>(f, num_sms, stream);
    }
    if (nvec <= 32 * 4) return launch_team<T, 1, 1, 4, 1, true>(f, (nvec + 31) / 32, num_sms, stream);
    if (nvec <= 128 * 2) return launch_forward<T, 4, 2, 2, true>(f, num_sms, stream);
    if (nvec <= 256 * 4) return launch_team<T, 8, 2, 4, 1, true>(f, (nvec + 255) / 256, num_sms, stream);
    if (nvec <= 512 * 4) return launch_team<T, 16, 3, 4, 1, true>(f, (nvec + 511) / 512, num_sms, stream);
    // (64 registers a thread: some of a row goes through local memory, and no row is ahead)
    return launch_team<T, 32, 3, LNBWD_RESIDUAL_MAX_C / Vec<T>::N / 1024, 1, false>(f, (nvec + 1023) / 1024, num_sms, stream);
}

// ---------------------------------------------------------------- backward

// One row's statistics and sums.
struct RowTerms {
    float mean, rstd, mean_post, rstd_post;  // 0 and 1 where there are none
    float a, c;                              // mean(g) (0 for RMS) and mean(g n)
    float e, h;                              // likewise of post
};

__device__ __forceinline__ RowTerms row_terms(const ResidualNorm& a, int64_t r) {
    RowTerms q{0.f, 1.f, 0.f, 1.f, 0.f, 0.f, 0.f, 0.f};
    if (a.norm == LAYER) q.mean = a.mean[r];
    if (a.norm != NONE) q.rstd = a.rstd[r];
    if (a.mean_post) q.mean_post = a.mean_post[r];
    if (a.rstd_post) q.rstd_post = a.rstd_post[r];
    return q;
}

// Per vector: dx from dout, dresidual, residual (n: the normalised residual).
template <int N>
__device__ __forceinline__ void dx_of(const RowTerms& q, bool norm, const float (&dout)[N], const float (&dres)[N],
                                      const float (&res)[N], const float (&w)[N], float (&n)[N], float (&dx)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        n[i] = (res[i] - q.mean) * q.rstd;
        dx[i] = norm ? fmaf(q.rstd, fmaf(w[i], dout[i], -fmaf(n[i], q.c, q.a)), dres[i]) : dres[i];
    }
}

struct Backward {
    ResidualNorm a;
    float* sums;      // [rows][4]: a, c, e, h (two passes)
    float* partials;  // [row blocks][4][C]: dweight, dbias, sum dx z, sum dx
    float inv_c;
    int row_blocks;
    int team_warps, teams;  // warps of a team, teams of a block
};

// ---- one pass

// E pairs of columns to a thread, R rows at a time, WARPS warps to a block, RING requests of
// R rows on their way or in use.
template <typename T_, int E_, int R_, int WARPS_, int RING_>
struct RowsConfig {
    using T = T_;
    static constexpr int E = E_, R = R_, WARPS = WARPS_, RING = RING_;
    static constexpr int V = 2 * E / Vec<T>::N, THREADS = 32 * WARPS;
    static constexpr uint32_t PART = R * V * THREADS * 16u, SLOT = 4 * PART;
    static constexpr int SMEM = static_cast<int>(RING * SLOT);
    static constexpr int MAX_C = THREADS * 2 * E;
    static_assert(SMEM >= 4 * 2 * E * 4 * THREADS && SMEM <= 220 * 1024, "the ring holds the sums of every thread, a block the ring");
};

// 2 R sums over a team, in a fixed order, in every thread. The 2 R values of a lane are
// halved in number with every exchange while there are several (lane group j of the warp
// ends with value j), so that a warp sums four in six exchanges; the warps' sums of a
// value are then summed by every warp the same way. `slots`: 2 x [warps][2 R] of the
// team, which alternate, so that one barrier is enough.
template <int R>
struct TeamSums {
    static constexpr int K = 2 * R;
    float* slots;
    int warp, warps, team;
    int which = 0;
    __device__ void operator()(float (&s)[K]) {
        const int lane = static_cast<int>(threadIdx.x & 31);
        float v;
        if constexpr (K == 4) {
            const bool upper = lane & 16, odd = lane & 8;
            const float a = (upper ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, upper ? s[0] : s[2], 16);
            const float b = (upper ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, upper ? s[1] : s[3], 16);
            v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
        } else {
            const bool upper = lane & 16;
            v = (upper ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, upper ? s[0] : s[1], 16);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) {  // value j is lane group j's
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] = __shfl_sync(0xffffffffu, v, k * (32 / K));
            return;
        }
        float* at = slots + which;
        which ^= warps * K;
        if (lane % (32 / K) == 0) at[warp * K + lane / (32 / K)] = v;
        ptx::named_bar_sync(static_cast<uint32_t>(1 + team), static_cast<uint32_t>(32 * warps));
        v = lane < warps * K ? at[lane] : 0.f;  // value lane % K of warp lane / K
        if (lane + 32 < warps * K) v += at[lane + 32];
#pragma unroll
        for (int o = K; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = __shfl_sync(0xffffffffu, v, k);
    }
};

// A team of warps owns R rows at a time; a thread has the same columns of all of its rows
// (16-byte vectors, 32 warps apart), their weights and their sums in registers. The next
// rows are on their way into shared memory, each thread's vectors to places that only it
// reads (no barrier). MEAN, MEAN_POST: norm, post subtracts a mean (LAYER); without, their sums
// of g are not formed (8192 x 1600 bf16 with two RMS norms takes 4 us less so). The columns' sums are
// fp32, a chain of a team's rows each: 777 x 1004 fp32 ends 1.5e-7 from the exact gradients
// where sums in 64 bits end 0.9e-7 from them, but 64 bits would double the four sums a column
// that fill the registers, and run at a small part of the fp32 rate.
template <typename L, bool MEAN, bool MEAN_POST>
__global__ void __launch_bounds__(L::THREADS, 1) residual_rows_kernel(const __grid_constant__ Backward b) {
    using T = typename L::T;
    constexpr int H = Pairs<T>::H, V = L::V, E = L::E, R = L::R, THREADS = L::THREADS;
    constexpr uint32_t PART = L::PART, SLOT = L::SLOT;  // vector j of row k of tensor i of a slot: at i PART + (k V + j) 16 THREADS
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float slots[2 * L::WARPS * 2 * R];
    const ResidualNorm& a = b.a;
    const int warps = b.team_warps, teams = b.teams;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int team = warp / warps, wt = warp % warps, t = wt * 32 + lane;
    if (team >= teams) return;  // (the block's warps beyond whole teams; no block-wide barrier waits for them)
    const int nvec = a.C / Vec<T>::N;
    const bool norm = a.norm != NONE, post = a.post != NONE;
    const uint32_t mine = ptx::smem_u32(ring) + threadIdx.x * 16u;
    int at[V];  // the thread's vectors of a row
    bool on[V];
#pragma unroll
    for (int j = 0; j < V; ++j) at[j] = t + 32 * warps * j, on[j] = at[j] < nvec;
    // what is not there, a whole tensor or a vector beyond the row, is zero throughout
    const void* tensors[4] = {a.dout, a.residual, a.dresidual, a.branch};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (!tensors[i] || !on[j])
                for (int k = 0; k < L::RING * R; ++k)
                    ptx::sts128u(mine + (k / R) * SLOT + i * PART + (k % R * V + j) * (THREADS * 16), make_uint4(0u, 0u, 0u, 0u));
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R, first = (static_cast<int64_t>(blockIdx.x) * teams + team) * R;
    int64_t ahead = first;  // the next rows to request, into slot `into`
    uint32_t into = 0, from = 0;
    auto request = [&]() {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (ahead + k < a.rows) {
                const int64_t row = (ahead + k) * nvec;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!tensors[i]) continue;
                    const uint4* p = static_cast<const uint4*>(tensors[i]) + row;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (on[j]) copy16(mine + into + i * PART + (k * V + j) * (THREADS * 16), p + at[j]);
                }
            }
        }
        copies_commit();
        ahead += step;
        into = into + SLOT == L::RING * SLOT ? 0 : into + SLOT;
    };
#pragma unroll
    for (int i = 0; i + 1 < L::RING; ++i) request();
    // the weights of a thread's columns, 0 beyond the row: nothing there adds to a sum
    F2 w[E], gw[E], s[4][E];  // gw: scale * gate * weight_post
#pragma unroll
    for (int j = 0; j < V; ++j) {
        auto column = [&](const void* p, float fill, F2 (&f)[H]) {
            if (on[j] && p) Pairs<T>::get(__ldg(static_cast<const uint4*>(p) + at[j]), f);
#pragma unroll
            for (int i = 0; i < H; ++i)
                if (!on[j] || !p) f[i] = F2::both(on[j] ? fill : 0.f);
        };
        F2 f[H], g[H];
        column(a.weight, 0.f, f);
#pragma unroll
        for (int i = 0; i < H; ++i) w[j * H + i] = f[i];
        column(a.gate, 1.f, g);
        column(a.weight_post, 1.f, f);
#pragma unroll
        for (int i = 0; i < H; ++i) gw[j * H + i] = mul2(mul2(F2::both(a.scale), g[i]), f[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) s[k][i] = F2::both(0.f);
    TeamSums<R> sums{slots + team * (4 * R * warps), wt, warps, team};
    RowTerms q[R], next[R];
    auto terms = [&](RowTerms (&to)[R], int64_t r) {
#pragma unroll
        for (int k = 0; k < R; ++k) to[k] = row_terms(a, min(r + k, a.rows - 1));
    };
    if (first < a.rows) terms(q, first);
    for (int64_t r = first; r < a.rows; r += step) {
        if (r + step < a.rows) terms(next, r + step);
        copies_wait_but<L::RING - 2>();
        request();  // into the slot of the rows before these
        bool there[R];  // (a row beyond the last: nothing of it is stored or summed)
#pragma unroll
        for (int k = 0; k < R; ++k) there[k] = k == 0 || r + k < a.rows;
        auto take = [&](int i, int k, F2 (&f)[E]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint4 v = ptx::lds128(mine + from + i * PART + (k * V + j) * (THREADS * 16));
                Pairs<T>::get(there[k] ? v : make_uint4(0u, 0u, 0u, 0u), f + j * H);
            }
        };
        auto put = [&](void* p, int k, const F2 (&f)[E]) {
            uint4* row = static_cast<uint4*>(p) + (r + k) * nvec;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (on[j] && there[k]) row[at[j]] = Pairs<T>::put(f + j * H);
        };
        F2 dx[R][E];
        float both[2 * R];
        if (norm) {
            F2 n[R][E], g[R][E];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                take(0, k, g[k]);
                take(1, k, n[k]);
                F2 s0 = F2::both(0.f), s1 = F2::both(0.f);
                const F2 m = F2::both(-q[k].mean), rstd = F2::both(q[k].rstd);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    n[k][i] = mul2(MEAN ? add2(n[k][i], m) : n[k][i], rstd);
                    s[0][i] = fma2(g[k][i], n[k][i], s[0][i]);
                    if (MEAN) s[1][i] = add2(s[1][i], g[k][i]);
                    g[k][i] = mul2(g[k][i], w[i]);
                    if (MEAN) s0 = add2(s0, g[k][i]);
                    s1 = fma2(g[k][i], n[k][i], s1);
                }
                both[2 * k] = s0.lo() + s0.hi(), both[2 * k + 1] = s1.lo() + s1.hi();
            }
            sums(both);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const F2 m = F2::both(-both[2 * k] * b.inv_c), c = F2::both(-both[2 * k + 1] * b.inv_c), rstd = F2::both(q[k].rstd);
                take(2, k, dx[k]);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const F2 d = fma2(n[k][i], c, g[k][i]);
                    dx[k][i] = fma2(rstd, MEAN ? add2(d, m) : d, dx[k][i]);
                }
                put(a.dx, k, dx[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                take(2, k, dx[k]);
                put(a.dx, k, dx[k]);
            }
        }
        F2 z[R][E];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            take(3, k, z[k]);
            F2 s0 = F2::both(0.f), s1 = F2::both(0.f);
            const F2 m = F2::both(-q[k].mean_post), rstd = F2::both(q[k].rstd_post);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (post) z[k][i] = mul2(MEAN_POST ? add2(z[k][i], m) : z[k][i], rstd);
                s[2][i] = fma2(dx[k][i], z[k][i], s[2][i]);
                if (MEAN_POST) s[3][i] = add2(s[3][i], dx[k][i]);
                dx[k][i] = mul2(gw[i], dx[k][i]);
                if (MEAN_POST) s0 = add2(s0, dx[k][i]);
                s1 = fma2(dx[k][i], z[k][i], s1);
            }
            both[2 * k] = s0.lo() + s0.hi(), both[2 * k + 1] = s1.lo() + s1.hi();
        }
        from = from + SLOT == L::RING * SLOT ? 0 : from + SLOT;
        if (a.dbranch) {
            if (post) {
                sums(both);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const F2 m = F2::both(-both[2 * k] * b.inv_c), c = F2::both(-both[2 * k + 1] * b.inv_c), rstd = F2::both(q[k].rstd_post);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const F2 d = fma2(z[k][i], c, dx[k][i]);
                        dx[k][i] = mul2(rstd, MEAN_POST ? add2(d, m) : d);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) put(a.dbranch, k, dx[k]);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) q[k] = next[k];
    }

    // The block's sums over its rows: the teams' in team order, through the ring's memory, where
    // value quad q of thread t of a team is at q * team + t.
    const int team_threads = 32 * warps, live = teams * team_threads;
    float* to = b.partials + static_cast<int64_t>(blockIdx.x) * 4 * a.C;
    auto column = [&](int quad, int thread) {  // of the quad's first value
        const int i = quad % (E / 2) * 2;
        return (thread + team_threads * (i / H)) * Vec<T>::N + 2 * (i % H);
    };
    copies_wait_but<0>();
    float4* joined = reinterpret_cast<float4*>(ring);
    if (teams > 1) ptx::named_bar_sync(0, static_cast<uint32_t>(live));
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const int quad = (f * E + i) / 2, c = column(quad, t);
            const float4 v = make_float4(s[f][i].lo(), s[f][i].hi(), s[f][i + 1].lo(), s[f][i + 1].hi());
            if (teams > 1) joined[(team * 2 * E + quad) * team_threads + t] = v;
            else if (c < a.C) *reinterpret_cast<float4*>(to + static_cast<int64_t>(f) * a.C + c) = v;
        }
    if (teams == 1) return;
    ptx::named_bar_sync(0, static_cast<uint32_t>(live));
    for (int k = static_cast<int>(threadIdx.x); k < 2 * E * team_threads; k += live) {
        const int quad = k / team_threads, c = column(quad, k % team_threads);
        if (c >= a.C) continue;
        float4 v = joined[k];
        for (int m = 1; m < teams; ++m) {
            const float4 u = joined[m * 2 * E * team_threads + k];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4*>(to + static_cast<int64_t>(quad / (E / 2)) * a.C + c) = v;
    }
}

template <typename T>
using NarrowRows = RowsConfig<T, 4, sizeof(T) == 2 ? 2 : 1, 16, 3>;  // up to 4096 columns
template <typename T>
using WideRows = RowsConfig<T, 8, 1, 12, sizeof(T) == 2 ? 3 : 2>;    // up to 6144
// Up to 8192, bf16 (the ring of fp32 rows does not fit): 128 registers a thread, a few of
// which go through local memory; 2000 x 8192 with two RMS norms 63 us, with two LayerNorms 90, in
// two passes 92 and 93.
using WidestRows = RowsConfig<__nv_bfloat16, 8, 1, 16, 3>;

template <typename L, bool MEAN, bool MEAN_POST>
cudaError_t launch_rows(const Backward& b, cudaLaunchConfig_t cfg) {
    constexpr auto kernel = residual_rows_kernel<L, MEAN, MEAN_POST>;
    cfg.gridDim = dim3(static_cast<unsigned>(b.row_blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(L::THREADS), 1, 1);
    cfg.dynamicSmemBytes = L::SMEM;
    const cudaError_t e = allow_smem<kernel>(L::SMEM);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, b) : e;
}

template <typename L>
cudaError_t launch_rows(const Backward& b, const cudaLaunchConfig_t& cfg) {
    if (b.a.norm == LAYER) return b.a.post == LAYER ? launch_rows<L, true, true>(b, cfg) : launch_rows<L, true, false>(b, cfg);
    return b.a.post == LAYER ? launch_rows<L, false, true>(b, cfg) : launch_rows<L, false, false>(b, cfg);
}

// ---- two passes

constexpr int SUM_THREADS = 256;

__device__ __forceinline__ float block_sum(float s, float* slots) {
    s = warp_sum(s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = slots[0];
#pragma unroll
    for (int w = 1; w < SUM_THREADS / 32; ++w) t += slots[w];
    return t;
}

template <typename T>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float (&f)[Vec<T>::N]) {
    if (p) {
        Vec<T>::get(reinterpret_cast<const uint4*>(p)[at], f);
    } else {
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) f[e] = 0.f;
    }
}

// A block per row: the sums that dx and dbranch need.
template <typename T>
__global__ void __launch_bounds__(SUM_THREADS) residual_sums_kernel(const __grid_constant__ Backward b) {
    using V = Vec<T>;
    constexpr int N = V::N;
    __shared__ float slots[SUM_THREADS / 32];
    const ResidualNorm& a = b.a;
    const int nvec = a.C / N;
    const bool norm = a.norm != NONE, post = a.post != NONE && a.dbranch;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        RowTerms q = row_terms(a, r);
        const int64_t at = r * nvec;
        if (norm) {
            float s0 = 0.f, s1 = 0.f;
            for (int v = static_cast<int>(threadIdx.x); v < nvec; v += SUM_THREADS) {
                float d[N], x[N], w[N];
                load_row<T>(a.dout, at + v, d);
                load_row<T>(a.residual, at + v, x);
                column<T>(a.weight, v, 1.f, w);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float g = w[i] * d[i];
                    s0 += g;
                    s1 = fmaf(g, (x[i] - q.mean) * q.rstd, s1);
                }
            }
            s0 = block_sum(s0, slots), s1 = block_sum(s1, slots);
            q.a = a.norm == LAYER ? s0 * b.inv_c : 0.f;
            q.c = s1 * b.inv_c;
        }
        if (post) {
            float s0 = 0.f, s1 = 0.f;
            for (int v = static_cast<int>(threadIdx.x); v < nvec; v += SUM_THREADS) {
                float d[N], x[N], w[N], dr[N], z[N], wp[N], g[N], n[N], dx[N];
                load_row<T>(norm ? a.dout : nullptr, at + v, d);
                load_row<T>(norm ? a.residual : nullptr, at + v, x);
                load_row<T>(a.dresidual, at + v, dr);
                load_row<T>(a.branch, at + v, z);
                column<T>(norm ? a.weight : nullptr, v, 1.f, w);
                column<T>(a.weight_post, v, 1.f, wp);
                column<T>(a.gate, v, 1.f, g);
                dx_of<N>(q, norm, d, dr, x, w, n, dx);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float y = a.scale * g[i] * wp[i] * dx[i];
                    s0 += y;
                    s1 = fmaf(y, (z[i] - q.mean_post) * q.rstd_post, s1);
                }
            }
            s0 = block_sum(s0, slots), s1 = block_sum(s1, slots);
            q.e = a.post == LAYER ? s0 * b.inv_c : 0.f;
            q.h = s1 * b.inv_c;
        }
        if (threadIdx.x == 0) reinterpret_cast<float4*>(b.sums)[r] = make_float4(q.a, q.c, q.e, q.h);
    }
}

constexpr int COL_THREADS = 128;

// A thread per vector of columns over a range of rows: dx, dbranch, and the columns' sums.
template <typename T>
__global__ void __launch_bounds__(COL_THREADS) residual_cols_kernel(const __grid_constant__ Backward b) {
    using V = Vec<T>;
    constexpr int N = V::N;
    const ResidualNorm& a = b.a;
    const int nvec = a.C / N;
    const int v = static_cast<int>(blockIdx.x) * COL_THREADS + static_cast<int>(threadIdx.x);
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if (v >= nvec) return;
    const bool norm = a.norm != NONE, post = a.post != NONE;
    const bool branch = (post && (a.dbranch || a.dweight_post)) || a.dgate;
    const int64_t r0 = a.rows * blockIdx.y / gridDim.y, r1 = a.rows * (blockIdx.y + 1) / gridDim.y;
    float w[N], wp[N], g[N], s[4][N];
    column<T>(norm ? a.weight : nullptr, v, 1.f, w);
    column<T>(post ? a.weight_post : nullptr, v, 1.f, wp);
    column<T>(a.gate, v, 1.f, g);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        g[i] *= a.scale;
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k][i] = 0.f;
    }
    for (int64_t r = r0; r < r1; ++r) {
        RowTerms q = row_terms(a, r);
        const float4 f = __ldcg(reinterpret_cast<const float4*>(b.sums) + r);
        q.a = f.x, q.c = f.y, q.e = f.z, q.h = f.w;
        const int64_t at = r * nvec + v;
        float d[N], x[N], dr[N], z[N], n[N], dx[N];
        load_row<T>(norm ? a.dout : nullptr, at, d);
        load_row<T>(norm ? a.residual : nullptr, at, x);
        load_row<T>(a.dresidual, at, dr);
        load_row<T>(branch ? a.branch : nullptr, at, z);
        dx_of<N>(q, norm, d, dr, x, w, n, dx);
        reinterpret_cast<uint4*>(a.dx)[at] = V::put(dx);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] = (z[i] - q.mean_post) * q.rstd_post;
            s[0][i] = fmaf(d[i], n[i], s[0][i]);
            s[1][i] += d[i];
            s[2][i] = fmaf(dx[i], z[i], s[2][i]);
            s[3][i] += dx[i];
        }
        if (a.dbranch) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float y = g[i] * dx[i];
                dx[i] = post ? q.rstd_post * fmaf(wp[i], y, -fmaf(z[i], q.h, q.e)) : y;
            }
            reinterpret_cast<uint4*>(a.dbranch)[at] = V::put(dx);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float4* to = reinterpret_cast<float4*>(b.partials + (static_cast<int64_t>(blockIdx.y) * 4 + k) * a.C + static_cast<int64_t>(v) * N);
#pragma unroll
        for (int i = 0; i < N; i += 4) to[i / 4] = make_float4(s[k][i], s[k][i + 1], s[k][i + 2], s[k][i + 3]);
    }
}

constexpr int PARAM_WARPS = 32;

// The partial sums of a column in block order, then the parameters' gradients:
// with Z = sum dx z and D = sum dx, dweight_post = scale gate Z, dbias_post = scale gate D and
// dgate = scale (weight_post Z + bias_post D). All that is latency: the warps share the row
// blocks, a batch of loads each, and the old gradients are on their way meanwhile (16 warps
// and one after the other, 8192 x 1600 bf16 took 37.3 us in all instead of 33.9, 777 x 1004
// fp32 13.0 instead of 10.6; 8 columns to a block instead of 32 35.1 and 11.7).
template <typename T>
__global__ void __launch_bounds__(32 * PARAM_WARPS) residual_params_kernel(const __grid_constant__ Backward b) {
    __shared__ float part[PARAM_WARPS][4][32];
    const ResidualNorm& a = b.a;
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const bool post = a.post != NONE;
    const T* const columns[3] = {static_cast<const T*>(a.gate), static_cast<const T*>(post ? a.weight_post : nullptr),
                                 static_cast<const T*>(a.post == LAYER ? a.bias_post : nullptr)};
    T* const grads[5] = {static_cast<T*>(a.norm != NONE ? a.dweight : nullptr), static_cast<T*>(a.norm == LAYER ? a.dbias : nullptr),
                         static_cast<T*>(a.gate ? a.dgate : nullptr), static_cast<T*>(post ? a.dweight_post : nullptr),
                         static_cast<T*>(a.post == LAYER ? a.dbias_post : nullptr)};
    float column[3] = {1.f, 1.f, 0.f}, old[5] = {};
    if (warp == 0 && c < a.C) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (columns[i]) column[i] = static_cast<float>(columns[i][c]);
#pragma unroll
        for (int i = 0; i < 5; ++i)
            if (grads[i]) old[i] = static_cast<float>(grads[i][c]);
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.C) {
        const int lo = b.row_blocks * warp / PARAM_WARPS, hi = b.row_blocks * (warp + 1) / PARAM_WARPS;
        for (int k = lo; k < hi; k += 8) {  // 32 loads in flight, added in order
            float v[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float* p = b.partials + static_cast<int64_t>(k + u) * 4 * a.C + c;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[u][i] = k + u < hi ? __ldcg(p + static_cast<int64_t>(i) * a.C) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] += v[u][i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][i][lane] = s[i];
    __syncthreads();
    if (warp < 4) {  // a sum each
        float t = part[0][warp][lane];
#pragma unroll
        for (int w = 1; w < PARAM_WARPS; ++w) t += part[w][warp][lane];
        part[0][warp][lane] = t;
    }
    __syncthreads();
    if (warp != 0 || c >= a.C) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = part[0][i][lane];
    const float g = a.scale * column[0];
    const float terms[5] = {s[0], s[1], a.scale * fmaf(column[1], s[2], column[2] * s[3]), g * s[2], g * s[3]};
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (grads[i]) grads[i][c] = static_cast<T>(old[i] + terms[i]);
}

constexpr int MAX_SMS = 152;  // of a full GB300; the workspace does not depend on the device

enum class Rows { NARROW, WIDE, WIDEST, TWO_PASSES };
Rows rows_of(int64_t C, int dtype) {
    if (C <= NarrowRows<float>::MAX_C) return Rows::NARROW;
    if (C <= WideRows<float>::MAX_C) return Rows::WIDE;
    return C <= WidestRows::MAX_C && dtype == MMBWD_BF16 ? Rows::WIDEST : Rows::TWO_PASSES;
}
static_assert(NarrowRows<float>::MAX_C == NarrowRows<__nv_bfloat16>::MAX_C && WideRows<float>::MAX_C == WideRows<__nv_bfloat16>::MAX_C);

// Warps of a team in one pass.
int team_warps_of(int64_t C, int dtype) {
    const int64_t per_warp = 64 * (rows_of(C, dtype) == Rows::NARROW ? NarrowRows<float>::E : WideRows<float>::E);
    return static_cast<int>((C + per_warp - 1) / per_warp);
}

// Rows that a team has at once, and teams of a block: as few as take the rows in one round
// over all SMs, up to what the block's warps give (with all of them 2364 x 80 bf16 took 11.5 us
// instead of 6.7, 57 x 144 9.7 instead of 5.3).
int rows_at_once(int64_t C, int dtype) {
    return rows_of(C, dtype) == Rows::NARROW && dtype == MMBWD_BF16 ? NarrowRows<__nv_bfloat16>::R : 1;
}
int teams_of(int64_t rows, int64_t C, int dtype) {
    if (rows_of(C, dtype) != Rows::NARROW) return 1;
    const int64_t a_round = static_cast<int64_t>(MAX_SMS) * rows_at_once(C, dtype);
    return static_cast<int>(std::min<int64_t>((rows + a_round - 1) / a_round, NarrowRows<float>::WARPS / team_warps_of(C, dtype)));
}

int row_blocks_of(int64_t rows, int64_t C, int dtype) {
    if (rows_of(C, dtype) != Rows::TWO_PASSES) {
        const int64_t at_once = static_cast<int64_t>(teams_of(rows, C, dtype)) * rows_at_once(C, dtype);
        return static_cast<int>(std::min<int64_t>((rows + at_once - 1) / at_once, MAX_SMS));
    }
    const int64_t nvec = C / (dtype == MMBWD_F32 ? 4 : 8), tiles = (nvec + COL_THREADS - 1) / COL_THREADS;
    // some eight blocks of a column tile to an SM
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, MAX_SMS * 8 / tiles)));
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t sums_bytes(int64_t rows, int64_t C, int dtype) { return rows_of(C, dtype) != Rows::TWO_PASSES ? 0 : align256(static_cast<size_t>(rows) * 16); }

template <typename T>
cudaError_t backward(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream) {
    Backward b{a, a.ws, a.ws + sums_bytes(a.rows, a.C, dtype) / 4, 1.f / static_cast<float>(a.C), row_blocks_of(a.rows, a.C, dtype), team_warps_of(a.C, dtype), teams_of(a.rows, a.C, dtype)};
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cudaError_t e;
    const Rows how = rows_of(a.C, dtype);
    if (how != Rows::TWO_PASSES) {
        b.row_blocks = std::min(b.row_blocks, num_sms);
        e = how == Rows::NARROW ? launch_rows<NarrowRows<T>>(b, cfg)
            : how == Rows::WIDE ? launch_rows<WideRows<T>>(b, cfg)
                                : launch_rows<WidestRows>(b, cfg);
    } else {
        cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, MAX_SMS * 8)), 1, 1);
        cfg.blockDim = dim3(SUM_THREADS, 1, 1);
        e = cudaLaunchKernelEx(&cfg, residual_sums_kernel<T>, b);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(static_cast<unsigned>((a.C / Vec<T>::N + COL_THREADS - 1) / COL_THREADS), static_cast<unsigned>(b.row_blocks), 1);
        cfg.blockDim = dim3(COL_THREADS, 1, 1);
        e = cudaLaunchKernelEx(&cfg, residual_cols_kernel<T>, b);
    }
    if (e != cudaSuccess) return e;
    const bool any = a.dgate || a.dweight_post || a.dbias_post || a.dweight || a.dbias;
    if (!any) return e;
    cfg.gridDim = dim3(static_cast<unsigned>((a.C + 31) / 32), 1, 1);
    cfg.blockDim = dim3(32 * PARAM_WARPS, 1, 1);
    return cudaLaunchKernelEx(&cfg, residual_params_kernel<T>, b);
}

}  // namespace

size_t residual_backward_workspace(int64_t rows, int64_t C, int dtype) {
    return sums_bytes(rows, C, dtype) +
           align256(static_cast<size_t>(row_blocks_of(rows, C, dtype)) * 4 * static_cast<size_t>(C) * 4);
}

cudaError_t residual_forward_launch(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    return dtype == MMBWD_F32 ? forward<float>(a, num_sms, stream) : forward<__nv_bfloat16>(a, num_sms, stream);
}

cudaError_t residual_backward_launch(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    return dtype == MMBWD_F32 ? backward<float>(a, dtype, num_sms, stream) : backward<__nv_bfloat16>(a, dtype, num_sms, stream);
}

}  // namespace mmbwd
