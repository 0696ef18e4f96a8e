// mmbwd_forward_act for few tokens (include/linear_epilogue.h): out (T x N) = act(inp (T x K) .
// weight (N x K)^T + bias) + residual, where the weight's bytes are the work.
//
// A warp streams a part of K of a few rows of the weight straight into registers, 16
// bytes a lane with the next loads always in flight, and multiplies it there. Where the
// rows alone give too few warps to keep HBM busy, several warps of a block share K and
// add their sums in warp order through shared memory. One launch, no workspace, the same
// bits on every call. Prompts of more tokens whose tiles of 32 x 32 run all at once go the same way.
//
// bf16: mma.sync with the tokens as its 16 rows and 8 rows of the weight as its columns.
// Which of a product's 16 values of k a lane holds does not matter as long as both
// operands agree: a lane's 16 bytes, k = 8 (lane % 4) .. + 7 of a 32-wide chunk, are
// the operands of two products, so neither operand is rearranged. (A tcgen05 tile of 128
// or 256 rows would be waited for and read back through tensor memory; at a token or a
// few the loads are all there is.)
// fp32: fused multiply-adds, a lane four values of k, four rows of the weight at a time.
#include "act.cuh"
#include "ops.h"
#include "ptx.cuh"

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cstring>

namespace mmbwd {
namespace {

constexpr int MAX_WARPS = 16;

struct Params {
    void *out, *pre;
    const void *inp, *weight, *bias, *residual;
    int64_t N, K;
    int T, act;
    int share;  // warps that share K, a power of two and at most the block's
};

// Two neighbouring outputs of a token: s = sum + bias, pre, act, residual.
template <typename T>
__device__ __forceinline__ void finish(const Params& p, int token, int64_t n, float s0, float s1) {
    constexpr bool FAST = sizeof(T) == 2;
    if (p.bias) {
        const T* b = static_cast<const T*>(p.bias) + n;
        s0 += static_cast<float>(b[0]), s1 += static_cast<float>(b[1]);
    }
    const int64_t at = token * p.N + n;
    auto store = [&](void* to, float a, float b) {
        if constexpr (FAST) *reinterpret_cast<__nv_bfloat162*>(static_cast<T*>(to) + at) = __floats2bfloat162_rn(a, b);
        else *reinterpret_cast<float2*>(static_cast<T*>(to) + at) = make_float2(a, b);
    };
    if (p.pre) store(p.pre, s0, s1);
    act::with(p.act, [&](auto kind) {
        constexpr int ACT = decltype(kind)::value;
        if constexpr (FAST) act::value_fast<ACT>(s0, s1);
        else s0 = act::value<ACT>(s0), s1 = act::value<ACT>(s1);
    });
    if (p.residual) {
        const T* r = static_cast<const T*>(p.residual) + at;
        s0 += static_cast<float>(r[0]), s1 += static_cast<float>(r[1]);
    }
    store(p.out, s0, s1);
}

// red[warp][TOKENS][ROWS]: the sums of each group of `share` warps in warp order, the outputs.
template <typename T, int TOKENS, int ROWS>
__device__ __forceinline__ void join(const Params& p, const float* red, int64_t n0, int t0, int tokens) {
    __syncthreads();
    const int groups = static_cast<int>(blockDim.x >> 5) / p.share, pairs = groups * tokens * (ROWS / 2);
    for (int e = static_cast<int>(threadIdx.x); e < pairs; e += static_cast<int>(blockDim.x)) {
        const int row = e % (ROWS / 2) * 2, rest = e / (ROWS / 2), group = rest % groups, token = rest / groups;
        const int64_t n = n0 + group * ROWS + row;
        if (n >= p.N) continue;
        const float* at = red + (group * p.share * TOKENS + token) * ROWS + row;
        float2 s = *reinterpret_cast<const float2*>(at);
        for (int w = 1; w < p.share; ++w) {
            const float2 v = *reinterpret_cast<const float2*>(at + w * TOKENS * ROWS);
            s.x += v.x, s.y += v.y;
        }
        finish<T>(p, t0 + token, n, s.x, s.y);
    }
}

__device__ __forceinline__ uint4 stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MT tiles of 16 tokens, NR groups of 8 weight rows to a warp, AHEAD chunks in flight.
template <int MT, int NR, int AHEAD, int WARPS = MAX_WARPS>
__global__ void __launch_bounds__(32 * WARPS) tokens_bf16_kernel(const __grid_constant__ Params p) {
    constexpr int ROWS = 8 * NR, TOKENS = 16 * MT;
    extern __shared__ __align__(16) float red[];  // [warp][TOKENS][ROWS]
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31), g = lane >> 2, t = lane & 3;
    const int group = warp / p.share, part = warp % p.share, groups = static_cast<int>(blockDim.x >> 5) / p.share;
    const int64_t block0 = static_cast<int64_t>(blockIdx.x) * (groups * ROWS), n0 = block0 + group * ROWS;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int t0 = static_cast<int>(blockIdx.y) * TOKENS, tokens = min(p.T - t0, TOKENS);
    // Rows beyond the last, and tokens, read the last one's: what they give is not stored.
    const __nv_bfloat16* w[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        w[i] = static_cast<const __nv_bfloat16*>(p.weight) + min(n0 + 8 * i + g, p.N - 1) * p.K + 8 * t;
    const __nv_bfloat16* x[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) x[i] = static_cast<const __nv_bfloat16*>(p.inp) + static_cast<int64_t>(t0 + min(8 * i + g, tokens - 1)) * p.K + 8 * t;
    float c[MT][NR][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[m][i][e] = 0.f;
    const int64_t chunks = (p.K + 31) / 32;
    const int lo = static_cast<int>(chunks * part / p.share), hi = static_cast<int>(chunks * (part + 1) / p.share);
    uint4 wv[AHEAD][NR], xv[AHEAD][2 * MT];
    auto fetch = [&](int u, int k) {
        const int64_t at = static_cast<int64_t>(k) * 32;
        const bool in = k < hi && at + 8 * t < p.K;  // (K is a multiple of 8)
#pragma unroll
        for (int i = 0; i < NR; ++i) wv[u][i] = in ? stream16(w[i] + at) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            xv[u][i] = in && (i == 0 || 8 * i < tokens) ? __ldg(reinterpret_cast<const uint4*>(x[i] + at)) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(u, lo + u);
    for (int k = lo; k < hi; k += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (k + u >= hi) break;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const uint4 &a = xv[u][2 * m], &b = xv[u][2 * m + 1], &v = wv[u][i];
                    mma(c[m][i], a.x, b.x, a.y, b.y, v.x, v.y);
                    mma(c[m][i], a.z, b.z, a.w, b.w, v.z, v.w);
                }
            fetch(u, k + u + AHEAD);
        }
    }
    if (p.share == 1) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int token = 16 * m + 8 * h + g;
                    const int64_t n = n0 + 8 * i + 2 * t;
                    if (token < tokens && n < p.N) finish<__nv_bfloat16>(p, t0 + token, n, c[m][i][2 * h], c[m][i][2 * h + 1]);
                }
        return;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (16 * m + 8 * h + g < tokens)
                    *reinterpret_cast<float2*>(red + (warp * TOKENS + 16 * m + 8 * h + g) * ROWS + 8 * i + 2 * t) =
                        make_float2(c[m][i][2 * h], c[m][i][2 * h + 1]);
    join<__nv_bfloat16, TOKENS, ROWS>(p, red, block0, t0, tokens);
}

// TOKENS tokens from blockIdx.y on (those beyond T read the last one's), four weight rows to
// a warp.
template <int TOKENS, int AHEAD>
__global__ void __launch_bounds__(32 * MAX_WARPS) tokens_f32_kernel(const __grid_constant__ Params p) {
    constexpr int ROWS = 4;
    extern __shared__ __align__(16) float red[];  // [warp][TOKENS][ROWS]
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int group = warp / p.share, part = warp % p.share, groups = static_cast<int>(blockDim.x >> 5) / p.share;
    const int64_t block0 = static_cast<int64_t>(blockIdx.x) * (groups * ROWS);
    const int64_t n0 = min(block0 + group * ROWS, p.N - ROWS);  // (N is a multiple of 4; a group beyond the last repeats it)
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float* w = static_cast<const float*>(p.weight) + n0 * p.K + 4 * lane;
    const int t0 = static_cast<int>(blockIdx.y) * TOKENS, tokens = min(p.T - t0, TOKENS);
    const float* x = static_cast<const float*>(p.inp) + static_cast<int64_t>(t0) * p.K + 4 * lane;
    float c[TOKENS][ROWS];
#pragma unroll
    for (int m = 0; m < TOKENS; ++m)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) c[m][i] = 0.f;
    const int64_t chunks = (p.K + 127) / 128;
    const int lo = static_cast<int>(chunks * part / p.share), hi = static_cast<int>(chunks * (part + 1) / p.share);
    uint4 wv[AHEAD][ROWS], xv[AHEAD][TOKENS];
    auto fetch = [&](int u, int k) {
        const int64_t at = static_cast<int64_t>(k) * 128;
        const bool in = k < hi && at + 4 * lane < p.K;  // (K is a multiple of 4)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) wv[u][i] = in ? stream16(w + i * p.K + at) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < TOKENS; ++m)
            xv[u][m] = in ? __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(min(m, tokens - 1)) * p.K + at)) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(u, lo + u);
    for (int k = lo; k < hi; k += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (k + u >= hi) break;
#pragma unroll
            for (int m = 0; m < TOKENS; ++m)
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    c[m][i] = fmaf(__uint_as_float(xv[u][m].x), __uint_as_float(wv[u][i].x), c[m][i]);
                    c[m][i] = fmaf(__uint_as_float(xv[u][m].y), __uint_as_float(wv[u][i].y), c[m][i]);
                    c[m][i] = fmaf(__uint_as_float(xv[u][m].z), __uint_as_float(wv[u][i].z), c[m][i]);
                    c[m][i] = fmaf(__uint_as_float(xv[u][m].w), __uint_as_float(wv[u][i].w), c[m][i]);
                }
            fetch(u, k + u + AHEAD);
        }
    }
#pragma unroll
    for (int m = 0; m < TOKENS; ++m) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c[m][i] += __shfl_xor_sync(0xffffffffu, c[m][i], o);
        if (lane == m) *reinterpret_cast<float4*>(red + (warp * TOKENS + m) * ROWS) = make_float4(c[m][0], c[m][1], c[m][2], c[m][3]);
    }
    join<float, TOKENS, ROWS>(p, red, block0, t0, tokens);
}

// A kernel of TOKENS tokens by ROWS rows to a warp, eight warps to a block or as many as share
// K, MOST at most.
template <auto kernel, int TOKENS, int ROWS, int MOST = MAX_WARPS>
cudaError_t launch(Params p, int share, cudaStream_t stream) {
    static_assert(MOST * TOKENS * ROWS * 4 <= 48 * 1024, "the warps' sums fit the shared memory that needs no allowance");
    const int warps = std::max(share, 8);
    p.share = share;
    const int64_t per_block = static_cast<int64_t>(warps / share) * ROWS, blocks = (p.N + per_block - 1) / per_block;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((p.T + TOKENS - 1) / TOKENS), 1);
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(warps * TOKENS * ROWS * 4);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// More than 32 tokens: how many of a block's eight warps share the K of 32 tokens by 32 rows,
// so that all blocks run at once; 0 where they do not.
int prompt_share(int64_t T, int64_t N, int num_sms) {
    const int64_t tiles = (T + 31) / 32 * ((N + 31) / 32);
    int share = 8;
    while (share > 0 && tiles * share > 8 * num_sms) share /= 2;
    return share;
}

}  // namespace

// Up to 32 tokens, and more by the time of either kernel (us, fitted to the sizes below): this one
// goes by the chunks of K that a warp has, the tensor-core kernel by the k-blocks
// of its rounds of tiles. Measured, this / that: 65 tokens 600 -> 600 4.5 / 7.8, 119 tokens 1720 -> 536 6.2 /
// 12.7, 133 tokens 168 -> 240 3.8 / 5.7, 128 tokens 768 -> 768 4.5 / 8.4, 768 -> 2304 6.6 / 8.5, 1600 -> 6400 28
// / 12.8, 256 tokens 3000 -> 504 8.5 / 18.1, 512 tokens 768 -> 768 12.0 / 8.4, 4000 -> 400 16.2 / 21.7;
// 32 tokens 1600 -> 6400 10.1 / 14.0, 6400 -> 1600 10.5 / 36.1; 16
// tokens 768 -> 50304 16.6 / 29.3; one token 1600 -> 6400 5.6 / 14.7.
// MMBWD_ACT_BF16_PATH = "tokens" or "tiles" forces this kernel (up to the tokens that a grid
// holds) or the tensor-core one (tests, tuning).
bool tokens_act_takes_bf16(int64_t T, int64_t K, int64_t N, int num_sms) {
    if (const char* e = std::getenv("MMBWD_ACT_BF16_PATH")) {
        if (std::strcmp(e, "tokens") == 0) return T <= 32 * 65535;
        if (std::strcmp(e, "tiles") == 0) return false;
    }
    if (T <= 32) return true;
    const int share = prompt_share(T, N, num_sms);
    if (share == 0) return false;
    const int64_t chunks = ((K + 31) / 32 + share - 1) / share, tiles = (T + 255) / 256 * ((N + 255) / 256), pairs = num_sms / 2;
    const double a_chunk = share == 8 ? 0.45 : share == 4 ? 0.55 : share == 2 ? 0.7 : 1.0;
    return 3.2 + a_chunk * static_cast<double>(chunks) < 5.0 + 0.28 * static_cast<double>((tiles + pairs - 1) / pairs * ((K + 63) / 64));
}

// How many warps share K: as many as give the device `want` warps or more, with two chunks
// each (fp32: one). Measured, us: one token 1600 -> 6400 bf16 shared by 8 warps 5.6, by 4 7.6, by 1 20;
// 6400 -> 1600 by 16 7.0, by 8 9.3; 16 tokens 768 -> 50304 by 1 16.6, by 4 18.5; one token
// 6400 -> 1600 fp32 by 8 8.6, by 4 9.4; 8 tokens by 4 17.5, by 8 20.4.
cudaError_t tokens_act_launch(void* out, void* pre, const void* inp, const void* weight, const void* bias,
                              const void* residual, int64_t T, int64_t K, int64_t N, int act, int dtype, int num_sms,
                              cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    const Params p{out, pre, inp, weight, bias, residual, N, K, static_cast<int>(T), act, 1};
    auto shared_by = [&](int64_t groups, int64_t chunks, int64_t want) {
        int share = 1;
        while (share < MAX_WARPS && groups * share < want && 2 * share <= chunks) share *= 2;
        return share;
    };
    if (dtype == MMBWD_F32) {
        const int share = shared_by(N / 4 * ((T + 7) / 8), (K + 127) / 128, T <= 4 ? 2400 : 1600);
        if (T <= 1) return launch<tokens_f32_kernel<1, 2>, 1, 4>(p, share, stream);
        if (T <= 4) return launch<tokens_f32_kernel<4, 2>, 4, 4>(p, share, stream);
        return launch<tokens_f32_kernel<8, 1>, 8, 4>(p, share, stream);
    }
    if (T > 32) return launch<tokens_bf16_kernel<2, 4, 2, 8>, 32, 32, 8>(p, std::max(1, prompt_share(T, N, num_sms)), stream);
    const int share = shared_by((N + 15) / 16, (K + 31) / 32 / 2, T <= 16 ? 2400 : 1600);
    if (T <= 16)  // (fewer loads in flight to a warp leave the registers for more of them)
        return share < MAX_WARPS ? launch<tokens_bf16_kernel<1, 2, 2>, 16, 16>(p, share, stream)
                                 : launch<tokens_bf16_kernel<1, 2, 4>, 16, 16>(p, share, stream);
    return launch<tokens_bf16_kernel<2, 2, 3>, 32, 16>(p, share, stream);
}

}  // namespace mmbwd
