// fp32 products of mmbwd_forward_act and mmbwd_run_act (include/linear_epilogue.h) that are
// too small for the tensor-core kernel's tiles of 256 x 128: tiles of 64 x 64 or 32 x 32,
// whose K is shared by the G warps of a block.
//
// Bound by fp32 fused multiply-adds (128 a clock and SM) where the tiles fill the device,
// by the latency of a block's loads below that; sharing K inside a block
// shortens that chain without a second launch or a workspace. Each warp
// accumulates every G-th K-tile (of 8) in registers, 8 x 16 or 4 x 8 outputs a thread, in pairs
// (two multiply-adds to an instruction: 1000 x 1600 -> 1600 in tiles of 64 170 -> 141 us), and the
// warps' sums are added in warp order through shared memory, where the epilogue
// starts: the same bits on every call. Shared memory gives a warp 32 values a clock, so the
// outputs of a thread are as many as its registers hold (8 x 8 of 64 threads, behind a barrier
// of theirs: 141 us, 8 x 16 of one warp: 128; the multiply-add pipe is then busy for 62% of
// the time). The backward's two products share one launch.
#include "act.cuh"
#include "ops.h"
#include "ptx.cuh"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

namespace mmbwd {
namespace {

constexpr int BK = 8, PAD = 4, GROUP = 32;

// One product D (M x N, row-major) = A . B: A (M x K) row-major, or stored (K x M) where
// a_km; B (K x N) row-major, or stored (N x K) where b_nk.
struct Product {
    float* D = nullptr;
    const float *A = nullptr, *B = nullptr;
    int64_t M = 0, N = 0, K = 0;
    int tiles_n = 0, tiles = 0;
};

struct Params {
    Product first, second;
    const float* bias;         // forward
    const float* residual;     // forward; may be D
    float* pre;                // forward: stored; backward: read, may be D
    float* dbias;              // second product
    int act;
};

enum Epilogue { FORWARD, DPRE, DWEIGHT };

template <int TM, int G>
constexpr int smem_bytes() {
    constexpr int TILE = 8 * TM, staged = G * 4 * BK * (TILE + PAD), sums = G * TILE * TILE + G * TILE;
    return 4 * (staged > sums ? staged : sums);
}

template <int TM, int G, bool A_KM, bool B_NK, Epilogue EPI>
__device__ __forceinline__ void tile_product(const Params& p, const Product& q, int tile, float* smem) {
    constexpr int TILE = 8 * TM, TN = 2 * TM, LD = TILE + PAD, LOADS = TILE * BK / 4 / GROUP, H = TM / 4, W = TN / 4;
    const int group = static_cast<int>(threadIdx.x) / GROUP, tid = static_cast<int>(threadIdx.x) % GROUP;
    const int tx = tid % 4, ty = tid / 4;
    const int64_t m0 = static_cast<int64_t>(tile / q.tiles_n) * TILE, n0 = static_cast<int64_t>(tile % q.tiles_n) * TILE;
    float* As = smem + group * 4 * BK * LD;  // [2][BK][LD]
    float* Bs = As + 2 * BK * LD;
    const bool sums = EPI == DWEIGHT && p.dbias != nullptr && n0 == 0;

    float4 ra[LOADS], rb[LOADS];
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int i = tid + l * GROUP;
            if (A_KM) {
                const int64_t k = k0 + i / (TILE / 4), m = m0 + i % (TILE / 4) * 4;
                ra[l] = k < q.K && m < q.M ? *reinterpret_cast<const float4*>(q.A + k * q.M + m) : zero;
            } else {
                const int64_t m = m0 + i / 2, k = k0 + i % 2 * 4;
                ra[l] = m < q.M && k < q.K ? *reinterpret_cast<const float4*>(q.A + m * q.K + k) : zero;
            }
            if (B_NK) {
                const int64_t n = n0 + i / 2, k = k0 + i % 2 * 4;
                rb[l] = n < q.N && k < q.K ? *reinterpret_cast<const float4*>(q.B + n * q.K + k) : zero;
            } else {
                const int64_t k = k0 + i / (TILE / 4), n = n0 + i % (TILE / 4) * 4;
                rb[l] = k < q.K && n < q.N ? *reinterpret_cast<const float4*>(q.B + k * q.N + n) : zero;
            }
        }
    };
    auto put = [&](float* to, const float4& v, int i, bool across) {
        if (across) {
            float* at = to + i % 2 * 4 * LD + i / 2;
            at[0] = v.x, at[LD] = v.y, at[2 * LD] = v.z, at[3 * LD] = v.w;
        } else {
            *reinterpret_cast<float4*>(to + i / (TILE / 4) * LD + i % (TILE / 4) * 4) = v;
        }
    };
    auto store = [&](int buf) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            put(As + buf * BK * LD, ra[l], tid + l * GROUP, !A_KM);
            put(Bs + buf * BK * LD, rb[l], tid + l * GROUP, B_NK);
        }
    };
    act::Two acc[TM][TN / 2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[i][j] = act::Two::both(0.f);
    float colsum[TILE / GROUP] = {};

    const int64_t step = static_cast<int64_t>(G) * BK;
    int64_t k0 = static_cast<int64_t>(group) * BK;
    int buf = 0;
    if (k0 < q.K) {
        load(k0);
        store(0);
        __syncwarp();
    }
    for (; k0 < q.K; k0 += step, buf ^= 1) {
        if (k0 + step < q.K) load(k0 + step);
        const float *a_s = As + buf * BK * LD, *b_s = Bs + buf * BK * LD;
        if (sums) {
#pragma unroll
            for (int k = 0; k < BK; ++k)
#pragma unroll
                for (int i = 0; i < TILE / GROUP; ++i) colsum[i] += a_s[k * LD + i * GROUP + tid];
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float a[TM];
            act::Two b[TN / 2];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 av = *reinterpret_cast<const float4*>(a_s + k * LD + ty * 4 + 32 * h);
                a[4 * h] = av.x, a[4 * h + 1] = av.y, a[4 * h + 2] = av.z, a[4 * h + 3] = av.w;
            }
#pragma unroll
            for (int h = 0; h < W; ++h) {
                const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(b_s + k * LD + tx * 4 + 16 * h);
                b[2 * h].v = bv.x, b[2 * h + 1].v = bv.y;
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN / 2; ++j) acc[i][j] = act::fma(act::Two::both(a[i]), b[j], acc[i][j]);
        }
        if (k0 + step < q.K) store(buf ^ 1);
        __syncwarp();
    }

    __syncthreads();  // the staged tiles have been read: their memory takes the groups' sums
    float* part = smem + group * TILE * TILE;
    float* colsums = smem + G * TILE * TILE;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < W; ++h)
            *reinterpret_cast<float4*>(part + (ty * 4 + (i & 3) + (i >> 2) * 32) * TILE + tx * 4 + 16 * h) =
                make_float4(acc[i][2 * h].lo(), acc[i][2 * h].hi(), acc[i][2 * h + 1].lo(), acc[i][2 * h + 1].hi());
    if (sums) {
#pragma unroll
        for (int i = 0; i < TILE / GROUP; ++i) colsums[group * TILE + i * GROUP + tid] = colsum[i];
    }
    __syncthreads();
    for (int e = static_cast<int>(threadIdx.x); e < TILE * TILE / 4; e += G * GROUP) {
        const int row = e / (TILE / 4), col = e % (TILE / 4) * 4;
        const int64_t m = m0 + row, n = n0 + col;
        if (m >= q.M || n >= q.N) continue;  // N is a multiple of 4: a float4 is all in or all out
        float4 o = *reinterpret_cast<const float4*>(smem + row * TILE + col);
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(smem + k * TILE * TILE + row * TILE + col);
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        }
        const int64_t at = m * q.N + n;
        if constexpr (EPI == FORWARD) {
            if (p.bias) {
                const float4 b = *reinterpret_cast<const float4*>(p.bias + n);
                o.x += b.x, o.y += b.y, o.z += b.z, o.w += b.w;
            }
            if (p.pre) *reinterpret_cast<float4*>(p.pre + at) = o;
            act::with(p.act, [&](auto kind) {
                constexpr int ACT = decltype(kind)::value;
                o.x = act::value<ACT>(o.x), o.y = act::value<ACT>(o.y);
                o.z = act::value<ACT>(o.z), o.w = act::value<ACT>(o.w);
            });
        }
        const float* add = EPI == FORWARD ? p.residual : EPI == DWEIGHT ? q.D : nullptr;
        if (add) {
            const float4 r = *reinterpret_cast<const float4*>(add + at);
            o.x += r.x, o.y += r.y, o.z += r.z, o.w += r.w;
        }
        if constexpr (EPI == DPRE) {
            const float4 x = *reinterpret_cast<const float4*>(p.pre + at);
            act::with(p.act, [&](auto kind) {
                constexpr int ACT = decltype(kind)::value;
                o.x *= act::slope<ACT>(x.x), o.y *= act::slope<ACT>(x.y);
                o.z *= act::slope<ACT>(x.z), o.w *= act::slope<ACT>(x.w);
            });
        }
        *reinterpret_cast<float4*>(q.D + at) = o;
    }
    if (sums && threadIdx.x < TILE && m0 + threadIdx.x < q.M) {
        float s = colsums[threadIdx.x];
#pragma unroll
        for (int k = 1; k < G; ++k) s += colsums[k * TILE + threadIdx.x];
        p.dbias[m0 + threadIdx.x] = s;
    }
}

template <int TM, int G>
__global__ void __launch_bounds__(G* GROUP) small_forward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    tile_product<TM, G, false, true, FORWARD>(p, p.first, static_cast<int>(blockIdx.x), smem);
}

template <int TM, int G>
__global__ void __launch_bounds__(G* GROUP) small_backward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    // the tiles with the longer sums first: the others fill the gaps behind them
    int b = static_cast<int>(blockIdx.x);
    const bool first_first = p.first.K >= p.second.K;
    const int ahead = first_first ? p.first.tiles : p.second.tiles;
    const bool dweight = first_first == (b < ahead);
    if (b >= ahead) b -= ahead;
    if (dweight) tile_product<TM, G, true, false, DWEIGHT>(p, p.first, b, smem);
    else tile_product<TM, G, false, false, DPRE>(p, p.second, b, smem);
}

template <auto kernel>
cudaError_t launch(const Params& p, int blocks, int threads, int smem, cudaStream_t stream) {
    if (smem > 48 * 1024) {
        static bool done[64];  // (calls hold the library's lock)
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64 || !done[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) done[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

int64_t tiles_of(int64_t M, int64_t N, int tile) { return (M + tile - 1) / tile * ((N + tile - 1) / tile); }

Product product(float* D, const float* A, const float* B, int64_t M, int64_t N, int64_t K, int tile) {
    return {D, A, B, M, N, K, static_cast<int>((N + tile - 1) / tile), static_cast<int>(tiles_of(M, N, tile))};
}

}  // namespace

namespace {

// Time models (us), fitted to the measurements below; times (us) on one GB300:
//                         tokens  32 x 32  64 x 64  spans (forward | backward 32, 64, spans)
//    16 x 6400 -> 1600        29.1     86.7      149    149 | 98.3  120 60.1
//    40 x 1600 -> 6400                 51.9     43.8   47.1 |  117  163  154
//    64 x  768 ->  768         9.7     10.1     23.0   27.0 | 15.5 22.1 26.0
//   100 x  768 -> 2304               18.4     23.3   27.5 | 41.3 55.6 61.4
//   200 x  264 ->  388                6.9     11.8   17.5 |  9.6 14.6 19.1
//   333 x  772 -> 1300               26.2     23.7   28.5 | 46.6 44.0 39.2
//   500 x  768 ->  768               26.6     23.3   28.1 | 39.3 36.6 27.6
//  1000 x 1600 -> 1600                182      128     47 |  290  228   80
//  2048 x 1600 -> 2400                525      342     89 |  839  641  260
// A block of 32 x 32 outputs takes 0.0148 us per value of K alone on its SM and 0.0107 beside
// others, and as long as 60 values more for its first loads and its sums; one of 64 x 64
// 0.0265 and 0.0298, and 120 values more; below 64 values some warps have none. The tensor
// cores' items of 256 x 128 take 0.72 us a k-block of 32 and 4 for the epilogue, 7 for the
// launch and its first loads.
double small_us(int tile, const Product* q, int n, int num_sms) {
    double work = 0.0, longest = 0.0;
    for (int i = 0; i < n; ++i) {
        const double K = static_cast<double>(q[i].K), tiles = static_cast<double>(tiles_of(q[i].M, q[i].N, tile));
        work += tiles * (tile == 32 ? (std::max(K, 64.0) + 60.0) * 0.0107 : (std::max(K, 64.0) + 120.0) * 0.0298);
        longest = std::max(longest, K * (tile == 32 ? 0.0148 : 0.0265));
    }
    return 3.0 + std::max(work / num_sms, longest);
}

double spans_us(const Product* q, int n, int num_sms) {
    const double pairs = num_sms / 2;
    double work = 0.0, longest = 0.0, items = 0.0;
    for (int i = 0; i < n; ++i) {
        const double count = static_cast<double>((q[i].M + 255) / 256 * ((q[i].N + 127) / 128));
        const double item = 0.72 * static_cast<double>((q[i].K + 31) / 32) + 4.0;
        work += count * item, items += count;
        longest = std::max(longest, item);
    }
    // one product: whole rounds of equal items; two: the short ones fill the gaps
    return 7.0 + (n == 1 ? std::ceil(items / pairs) * longest : std::max(longest, work / pairs + 0.3 * longest));
}

// MMBWD_ACT_F32_PATH = "32", "64" or "spans" forces a kernel (tests, tuning).
ActPath fastest(const Product* q, int n, int num_sms) {
    if (const char* e = std::getenv("MMBWD_ACT_F32_PATH")) {
        if (std::strcmp(e, "32") == 0) return ActPath::SMALL_32;
        if (std::strcmp(e, "64") == 0) return ActPath::SMALL_64;
        if (std::strcmp(e, "spans") == 0) return ActPath::SPANS;
    }
    const double a = small_us(32, q, n, num_sms), b = small_us(64, q, n, num_sms), c = spans_us(q, n, num_sms);
    return c <= a && c <= b ? ActPath::SPANS : a <= b ? ActPath::SMALL_32 : ActPath::SMALL_64;
}

}  // namespace

ActPath act_forward_path(int64_t BT, int64_t C, int64_t OC, int num_sms) {
    const Product q = product(nullptr, nullptr, nullptr, BT, OC, C, 32);
    if (BT <= ACT_TOKENS && !std::getenv("MMBWD_ACT_F32_PATH")) {
        // a pass over the weight for every eight tokens
        const double tokens = 3.0 + static_cast<double>((BT + 7) / 8) * static_cast<double>(C) * static_cast<double>(OC) * 4.0 / 2.7e6;
        if (BT <= 8 || tokens <= std::min({small_us(32, &q, 1, num_sms), small_us(64, &q, 1, num_sms), spans_us(&q, 1, num_sms)}))
            return ActPath::TOKENS;
    }
    return fastest(&q, 1, num_sms);
}

ActPath act_run_path(int64_t BT, int64_t C, int64_t OC, int num_sms) {
    const Product q[2] = {product(nullptr, nullptr, nullptr, OC, C, BT, 32), product(nullptr, nullptr, nullptr, BT, C, OC, 32)};
    return fastest(q, 2, num_sms);
}

cudaError_t simt_small_forward_launch(int tile, float* out, float* pre, const float* inp, const float* weight,
                                      const float* bias, const float* residual, int64_t BT, int64_t C, int64_t OC,
                                      int act, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Params p{product(out, inp, weight, BT, OC, C, tile), {}, bias, residual, pre, nullptr, act};
    if (tile == 64) return launch<small_forward_kernel<8, 8>>(p, p.first.tiles, 8 * GROUP, smem_bytes<8, 8>(), stream);
    return launch<small_forward_kernel<4, 8>>(p, p.first.tiles, 8 * GROUP, smem_bytes<4, 8>(), stream);
}

cudaError_t simt_small_run_launch(int tile, float* dpre, float* dweight, float* dbias, const float* dout,
                                  const float* inp, const float* weight, const float* pre, int64_t BT, int64_t C,
                                  int64_t OC, int act, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Params p{product(dweight, dout, inp, OC, C, BT, tile), product(dpre, dout, weight, BT, C, OC, tile), nullptr, nullptr,
             const_cast<float*>(pre), dbias, act};
    const int blocks = p.first.tiles + p.second.tiles;
    if (tile == 64) return launch<small_backward_kernel<8, 8>>(p, blocks, 8 * GROUP, smem_bytes<8, 8>(), stream);
    return launch<small_backward_kernel<4, 8>>(p, blocks, 8 * GROUP, smem_bytes<4, 8>(), stream);
}

}  // namespace mmbwd
