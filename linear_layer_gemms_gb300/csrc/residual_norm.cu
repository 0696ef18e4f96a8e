// The step between two blocks (include/residual_norm.h): residual_out = x + scale * gate *
// post(branch), out = norm(residual_out), and its gradients.
//
// Bound by HBM. Forward: two rows read, two written. A team of P warps owns a row and
// keeps it in registers (VPT 16-byte vectors per thread) from the branch's statistics to
// the output, so nothing is read twice and each variance comes from the differences
// (LAYER) of values at hand. Backward: four rows read, two written. A team owns a row as
// well, a thread eight columns of it; it has the next row in flight, forms the row's
// four sums in two rounds and keeps its columns' parameter sums in registers over all
// rows of the team. Rows that no team of 16 warps holds (C > 4096) take two passes: one
// forms the rows' sums, one goes down column tiles.
#include "../../include/residual_norm.h"
#include "ops.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

namespace mmbwd {
namespace {

constexpr int NONE = LNBWD_NORM_NONE, LAYER = LNBWD_NORM_LAYER, RMS = LNBWD_NORM_RMS;

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

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The sum of a team's P warp sums, in warp order, in every thread. Consecutive sums
// alternate between two sets of slots, so that one barrier per sum is enough.
template <int P>
struct TeamSum {
    float* slots;  // 2 P floats
    int warp, team, which = 0;
    __device__ float operator()(float s) {
        s = warp_sum(s);
        if constexpr (P == 1) {
            return s;
        } else {
            float* at = slots + which * P;
            which ^= 1;
            if ((threadIdx.x & 31) == 0) at[warp] = s;
            ptx::named_bar_sync(static_cast<uint32_t>(1 + team), 32 * P);
            float t = at[0];
#pragma unroll
            for (int w = 1; w < P; ++w) t += at[w];
            return t;
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

template <int P>
constexpr int TEAMS = P == 1 ? 4 : 1;  // teams of one warp share a block of four rows

struct Forward {
    ResidualNorm a;
    float inv_c;
};

// Mean (0 without one) and rstd of the team's row, v[0 .. VPT N) in each thread; the
// values beyond the row are zero and `last` says whether the last vector is in it.
template <int KIND, int P, int N, int VPT>
__device__ __forceinline__ void statistics(const float (&v)[VPT * N], bool last, int C, float inv_c, float eps,
                                           TeamSum<P>& sum, float* mean, float* rstd) {
    float m = 0.f;
    if (KIND == LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT * N; ++i) s += v[i];
        m = mean_of(sum(s), C, inv_c);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT * N; ++i) {
        const float d = i < (VPT - 1) * N || last ? v[i] - m : 0.f;
        s = fmaf(d, d, s);
    }
    *mean = m;
    *rstd = 1.f / sqrtf(fmaf(sum(s), inv_c, eps));
}

template <typename T, int P, int VPT>
__global__ void __launch_bounds__(32 * P * TEAMS<P>) residual_forward_kernel(const __grid_constant__ Forward f) {
    using V = Vec<T>;
    constexpr int N = V::N;
    __shared__ float slots[TEAMS<P>][2 * P];
    const ResidualNorm& a = f.a;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int team = warp / P, wt = warp % P, t = wt * 32 + lane;
    const int nvec = a.C / N;
    const bool last = t + 32 * P * (VPT - 1) < nvec;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS<P> + team;
    if (r >= a.rows) return;
    TeamSum<P> sum{slots[team], wt, team};
    const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + r * a.C);
    const uint4* br = reinterpret_cast<const uint4*>(static_cast<const T*>(a.branch) + r * a.C);
    uint4 x[VPT];
    float v[VPT * N];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const bool on = j + 1 < VPT || last;
        x[j] = on ? xr[t + 32 * P * j] : make_uint4(0u, 0u, 0u, 0u);
        V::get(on ? br[t + 32 * P * j] : make_uint4(0u, 0u, 0u, 0u), v + j * N);
    }
    float mean = 0.f, rstd = 1.f;
    if (a.post != NONE) {
        if (a.post == LAYER) {
            statistics<LAYER, P, N, VPT>(v, last, a.C, f.inv_c, a.eps, sum, &mean, &rstd);
            if (a.mean_post && t == 0) a.mean_post[r] = mean;
        } else {
            statistics<RMS, P, N, VPT>(v, last, a.C, f.inv_c, a.eps, sum, &mean, &rstd);
        }
        if (a.rstd_post && t == 0) a.rstd_post[r] = rstd;
    }
    uint4* ro = reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + r * a.C);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + 32 * P * j;
        if (j + 1 < VPT || last) {
            float g[N], xv[N];
            V::get(x[j], xv);
            if (a.post != NONE) {
                float w[N], b[N];
                column<T>(a.weight_post, k, 1.f, w);
                column<T>(a.post == LAYER ? a.bias_post : nullptr, k, 0.f, b);
#pragma unroll
                for (int e = 0; e < N; ++e) v[j * N + e] = fmaf((v[j * N + e] - mean) * rstd, w[e], b[e]);
            }
            column<T>(a.gate, k, 1.f, g);
#pragma unroll
            for (int e = 0; e < N; ++e) v[j * N + e] = fmaf(a.scale * g[e], v[j * N + e], xv[e]);
            ro[k] = V::put(v + j * N);
        }
    }
    if (a.norm == NONE) return;
    if (a.norm == LAYER) {
        statistics<LAYER, P, N, VPT>(v, last, a.C, f.inv_c, a.eps, sum, &mean, &rstd);
        if (a.mean && t == 0) a.mean[r] = mean;
    } else {
        statistics<RMS, P, N, VPT>(v, last, a.C, f.inv_c, a.eps, sum, &mean, &rstd);
    }
    if (a.rstd && t == 0) a.rstd[r] = rstd;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + r * a.C);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + 32 * P * j;
        if (j + 1 < VPT || last) {
            float w[N], b[N];
            column<T>(a.weight, k, 1.f, w);
            column<T>(a.norm == LAYER ? a.bias : nullptr, k, 0.f, b);
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = fmaf((v[j * N + e] - mean) * rstd, w[e], b[e]);
            __stcs(o + k, V::put(w));
        }
    }
}

// The kernel whose team holds a row in exactly `need` vectors a thread, VPT to MOST.
template <typename T, int P, int VPT, int MOST>
cudaError_t launch_team(const Forward& f, int need, cudaStream_t stream) {
    if constexpr (VPT < MOST) {
        if (need > VPT) return launch_team<T, P, VPT + 1, MOST>(f, need, stream);
    }
    const int64_t blocks = (f.a.rows + TEAMS<P> - 1) / TEAMS<P>;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(32 * P * TEAMS<P>, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, residual_forward_kernel<T, P, VPT>, f);
}

template <typename T>
cudaError_t forward(const ResidualNorm& a, cudaStream_t stream) {
    const Forward f{a, 1.f / static_cast<float>(a.C)};
    const int nvec = a.C / Vec<T>::N;
    if (nvec <= 32 * 8) return launch_team<T, 1, 1, 8>(f, (nvec + 31) / 32, stream);
    if (nvec <= 128 * 4) return launch_team<T, 4, 3, 4>(f, (nvec + 127) / 128, stream);
    if (nvec <= 256 * 4) return launch_team<T, 8, 3, 4>(f, (nvec + 255) / 256, stream);
    if (nvec <= 512 * 4) return launch_team<T, 16, 3, 4>(f, (nvec + 511) / 512, stream);
    return launch_team<T, 32, 3, LNBWD_RESIDUAL_MAX_C / Vec<T>::N / 1024>(f, (nvec + 1023) / 1024, stream);
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
    int team_warps;   // one pass: warps of a team
    float inv_c;
    int row_blocks;
};

// ---- one pass

constexpr int COLS = 8;         // columns of a thread
constexpr int TEAM_WARPS = 16;  // warps of a block, at most

// A thread's eight values of a row, as they are stored.
template <typename T>
struct Eight {
    static constexpr int V = 8 / Vec<T>::N;
    uint4 v[V];
    // `p` at the row's first value; vector i is there if `on[i]`
    __device__ void load(const T* p, int c0, const bool (&on)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = p && on[i] ? reinterpret_cast<const uint4*>(p + c0)[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) Vec<T>::get(v[i], f + i * Vec<T>::N);
    }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, int c0, const bool (&on)[Eight<T>::V], const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < Eight<T>::V; ++i)
        if (on[i]) reinterpret_cast<uint4*>(p + c0)[i] = Vec<T>::put(f + i * Vec<T>::N);
}

// Two sums over a team, in warp order, in every thread; `at`: the team's slots. Consecutive
// sums of a team alternate between two sets of slots, so that one barrier is enough.
__device__ __forceinline__ float2 team_sum2(float x, float y, float2* at, int warp, int warps, int team) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (warps == 1) return make_float2(x, y);
    if ((threadIdx.x & 31) == 0) at[warp] = make_float2(x, y);
    ptx::named_bar_sync(static_cast<uint32_t>(1 + team), static_cast<uint32_t>(32 * warps));
    float2 t = at[0];
#pragma unroll
    for (int w = 1; w < TEAM_WARPS; ++w)
        if (w < warps) t.x += at[w].x, t.y += at[w].y;
    return t;
}

template <typename T>
struct RowData {
    Eight<T> dout, res, dres, branch;
    float mean, rstd, mean_post, rstd_post;
};

template <typename T>
__global__ void __launch_bounds__(32 * TEAM_WARPS, 1) residual_rows_kernel(const __grid_constant__ Backward b) {
    constexpr int V = Eight<T>::V;
    __shared__ float2 slots[TEAM_WARPS][2][TEAM_WARPS];
    __shared__ float joined[4 * 256 * (TEAM_WARPS / 2)];  // teams of at most half the warps are joined
    const ResidualNorm& a = b.a;
    const int warps = b.team_warps, warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int teams = static_cast<int>(blockDim.x >> 5) / warps, team = warp / warps, wt = warp % warps;
    const int c0 = (wt * 32 + lane) * COLS;
    bool on[V];
#pragma unroll
    for (int i = 0; i < V; ++i) on[i] = c0 + i * Vec<T>::N < a.C;
    const bool norm = a.norm != NONE, post = a.post != NONE;
    float2* at = slots[team][0];
    int which = 0;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    // the weights of a thread's columns, 0 beyond the row: nothing there adds to a sum
    float w[8], gw[8];  // gw: scale * gate * weight_post
    {
        Eight<T> t;
        t.load(static_cast<const T*>(a.weight), c0, on);
        t.get(w);
        t.load(static_cast<const T*>(a.weight_post), c0, on);
        t.get(gw);
        float g[8];
        t.load(static_cast<const T*>(a.gate), c0, on);
        t.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float one = on[i / Vec<T>::N] ? 1.f : 0.f;
            gw[i] = (post ? gw[i] : one) * (a.scale * (a.gate ? g[i] : one));
        }
    }
    float s[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[k][i] = 0.f;

    auto fetch = [&](RowData<T>& q, int64_t r) {
        const int64_t o = r * a.C;
        auto row = [&](const void* p) { return p ? static_cast<const T*>(p) + o : nullptr; };
        q.dout.load(row(a.dout), c0, on);
        q.res.load(row(a.residual), c0, on);
        q.dres.load(row(a.dresidual), c0, on);
        q.branch.load(row(a.branch), c0, on);
        const RowTerms t = row_terms(a, r);
        q.mean = t.mean, q.rstd = t.rstd, q.mean_post = t.mean_post, q.rstd_post = t.rstd_post;
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * teams;
    int64_t r = static_cast<int64_t>(blockIdx.x) * teams + team;
    RowData<T> q, next;
    if (r < a.rows) fetch(q, r);
    for (; r < a.rows; r += stride) {
        if (r + stride < a.rows) fetch(next, r + stride);
        float dx[8], z[8];
        q.dres.get(dx);
        if (norm) {
            float d[8], n[8], g[8], s0 = 0.f, s1 = 0.f;
            q.dout.get(d);
            q.res.get(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] = (n[i] - q.mean) * q.rstd;
                g[i] = w[i] * d[i];
                s0 += g[i];
                s1 = fmaf(g[i], n[i], s1);
                s[0][i] = fmaf(d[i], n[i], s[0][i]);
                s[1][i] += d[i];
            }
            const float2 t = team_sum2(s0, s1, at + which, wt, warps, team);
            which ^= TEAM_WARPS;
            const float m = a.norm == LAYER ? t.x * b.inv_c : 0.f, c = t.y * b.inv_c;
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] = fmaf(q.rstd, g[i] - fmaf(n[i], c, m), dx[i]);
        }
        store8(static_cast<T*>(a.dx) + r * a.C, c0, on, dx);
        q.branch.get(z);
        float y[8], s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = (z[i] - q.mean_post) * q.rstd_post;
            y[i] = gw[i] * dx[i];
            s0 += y[i];
            s1 = fmaf(y[i], z[i], s1);
            s[2][i] = fmaf(dx[i], z[i], s[2][i]);
            s[3][i] += dx[i];
        }
        if (a.dbranch) {
            if (post) {
                const float2 t = team_sum2(s0, s1, at + which, wt, warps, team);
                which ^= TEAM_WARPS;
                const float m = a.post == LAYER ? t.x * b.inv_c : 0.f, c = t.y * b.inv_c;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = q.rstd_post * (y[i] - fmaf(z[i], c, m));
            }
            store8(static_cast<T*>(a.dbranch) + r * a.C, c0, on, y);
        }
        q = next;
    }

    // The block's sums over its rows: the teams' in team order.
    float* to = b.partials + static_cast<int64_t>(blockIdx.x) * 4 * a.C;
    for (int k = 0; k < teams; ++k) {
        if (teams > 1) __syncthreads();
        if (team != k) continue;
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                float4 v = make_float4(s[f][i], s[f][i + 1], s[f][i + 2], s[f][i + 3]);
                if (teams > 1) {
                    float4* mine = reinterpret_cast<float4*>(joined + f * 256 * warps + c0 + i);
                    if (k > 0) v.x += mine->x, v.y += mine->y, v.z += mine->z, v.w += mine->w;
                    if (k + 1 < teams) *mine = v;
                }
                if (k + 1 == teams && c0 + i < a.C) *reinterpret_cast<float4*>(to + static_cast<int64_t>(f) * a.C + c0 + i) = v;
            }
    }
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

constexpr int PARAM_WARPS = 16;

// The partial sums of a column in block order, then the parameters' gradients:
// with Z = sum dx z and D = sum dx, dweight_post = scale gate Z, dbias_post = scale gate D and
// dgate = scale (weight_post Z + bias_post D).
template <typename T>
__global__ void __launch_bounds__(32 * PARAM_WARPS) residual_params_kernel(const __grid_constant__ Backward b) {
    __shared__ float part[PARAM_WARPS][4][32];
    const ResidualNorm& a = b.a;
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.C) {
        const int lo = b.row_blocks * warp / PARAM_WARPS, hi = b.row_blocks * (warp + 1) / PARAM_WARPS;
#pragma unroll 4
        for (int k = lo; k < hi; ++k) {
            const float* p = b.partials + static_cast<int64_t>(k) * 4 * a.C + c;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += __ldcg(p + static_cast<int64_t>(i) * a.C);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][i][lane] = s[i];
    __syncthreads();
    if (warp != 0 || c >= a.C) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] = part[0][i][lane];
#pragma unroll
        for (int w = 1; w < PARAM_WARPS; ++w) s[i] += part[w][i][lane];
    }
    auto at = [&](const void* p, float fill) { return p ? static_cast<float>(static_cast<const T*>(p)[c]) : fill; };
    auto add = [&](void* p, float x) {
        if (p) static_cast<T*>(p)[c] = static_cast<T>(static_cast<float>(static_cast<const T*>(p)[c]) + x);
    };
    const bool post = a.post != NONE;
    const float g = a.scale * at(a.gate, 1.f);
    if (a.norm != NONE) add(a.dweight, s[0]);
    if (a.norm == LAYER) add(a.dbias, s[1]);
    if (a.gate)
        add(a.dgate, a.scale * fmaf(at(post ? a.weight_post : nullptr, 1.f), s[2],
                                    at(a.post == LAYER ? a.bias_post : nullptr, 0.f) * s[3]));
    if (post) add(a.dweight_post, g * s[2]);
    if (a.post == LAYER) add(a.dbias_post, g * s[3]);
}

// Warps of a team in one pass; 0: two passes.
int team_warps_of(int64_t C) {
    const int64_t w = (C + 32 * COLS - 1) / (32 * COLS);
    return w <= TEAM_WARPS ? static_cast<int>(w) : 0;
}

constexpr int MAX_SMS = 152;  // of a full GB300; the workspace does not depend on the device

int row_blocks_of(int64_t rows, int64_t C, int dtype) {
    if (const int w = team_warps_of(C)) {
        const int64_t teams = TEAM_WARPS / w;
        return static_cast<int>(std::min<int64_t>((rows + teams - 1) / teams, MAX_SMS));
    }
    const int64_t nvec = C / (dtype == MMBWD_F32 ? 4 : 8), tiles = (nvec + COL_THREADS - 1) / COL_THREADS;
    // some eight blocks of a column tile to an SM
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, MAX_SMS * 8 / tiles)));
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t sums_bytes(int64_t rows, int64_t C) { return team_warps_of(C) ? 0 : align256(static_cast<size_t>(rows) * 16); }

template <typename T>
cudaError_t backward(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream) {
    Backward b{a, a.ws, a.ws + sums_bytes(a.rows, a.C) / 4, team_warps_of(a.C), 1.f / static_cast<float>(a.C),
               row_blocks_of(a.rows, a.C, dtype)};
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cudaError_t e;
    if (b.team_warps) {
        b.row_blocks = std::min(b.row_blocks, num_sms);
        cfg.gridDim = dim3(static_cast<unsigned>(b.row_blocks), 1, 1);
        cfg.blockDim = dim3(static_cast<unsigned>(32 * b.team_warps * (TEAM_WARPS / b.team_warps)), 1, 1);
        e = cudaLaunchKernelEx(&cfg, residual_rows_kernel<T>, b);
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
    return sums_bytes(rows, C) +
           align256(static_cast<size_t>(row_blocks_of(rows, C, dtype)) * 4 * static_cast<size_t>(C) * 4);
}

cudaError_t residual_forward_launch(const ResidualNorm& a, int dtype, int /*num_sms*/, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    return dtype == MMBWD_F32 ? forward<float>(a, stream) : forward<__nv_bfloat16>(a, stream);
}

cudaError_t residual_backward_launch(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    return dtype == MMBWD_F32 ? backward<float>(a, dtype, num_sms, stream) : backward<__nv_bfloat16>(a, dtype, num_sms, stream);
}

}  // namespace mmbwd
