// fp32 products of mmbwd_forward_act and mmbwd_run_act (include/linear_epilogue.h) that are
// too small for the tensor-core kernel's tiles of 256 x 128: tiles of 64 x 64 or 32 x 32,
// whose K is shared by the G warps of a block, and by the blocks of a cluster where the
// tiles are few.
//
// Bound by fp32 fused multiply-adds (128 a clock and SM) where the tiles fill the device,
// by the latency of a block's loads below that; sharing K inside a block
// shortens that chain without a second launch or a workspace. Each warp
// accumulates every G-th K-tile (of 8) in registers, 8 x 16 or 4 x 8 outputs a thread, in pairs
// (two multiply-adds to an instruction: 1000 x 1600 -> 1600 in tiles of 64 170 -> 141 us), and the
// warps' sums are added in warp order through shared memory, the blocks' in block order
// from one another's, where the epilogue starts: the same bits on every call. Shared memory gives a warp 32 values a clock, so the
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
    int share = 1;  // blocks (a whole cluster) that share K
    __host__ __device__ int blocks(int cluster) const { return (tiles * share + cluster - 1) / cluster * cluster; }
};

struct Params {
    Product first, second;
    const float* bias;         // forward
    const float* residual;     // forward; may be D
    float* pre;                // forward: stored, may be null; backward: read, may be D, null without an activation
    float* dbias;              // second product
    int act;
    int cluster;               // blocks of a cluster; a product is shared by all of them or by none
};

// Four values of shared memory anywhere in the cluster.
__device__ __forceinline__ float4 ld_cluster(const float* p, int rank) {
    const uint32_t at = ptx::mapa(ptx::smem_u32(p), static_cast<uint32_t>(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void add(float4& o, const float4& v) { o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w; }

enum Epilogue { FORWARD, DPRE, DWEIGHT };

template <int TM, int G>
constexpr int smem_bytes() {
    constexpr int TILE = 8 * TM, staged = G * 4 * BK * (TILE + PAD), sums = G * TILE * TILE + G * TILE;
    return 4 * (staged > sums ? staged : sums);
}

template <int TM, int G, bool A_KM, bool B_NK, Epilogue EPI>
__device__ __forceinline__ void tile_product(const Params& p, const Product& q, int tile, int rank, float* smem) {
    constexpr int TILE = 8 * TM, TN = 2 * TM, LD = TILE + PAD, LOADS = TILE * BK / 4 / GROUP, H = TM / 4, W = TN / 4;
    const int group = static_cast<int>(threadIdx.x) / GROUP, tid = static_cast<int>(threadIdx.x) % GROUP;
    const int tx = tid % 4, ty = tid / 4;
    const int64_t m0 = static_cast<int64_t>(tile / q.tiles_n) * TILE, n0 = static_cast<int64_t>(tile % q.tiles_n) * TILE;
    float* As = smem + group * 4 * BK * LD;  // [2][BK][LD]
    float* Bs = As + 2 * BK * LD;
    const bool sums = EPI == DWEIGHT && p.dbias != nullptr && n0 == 0;

    // What the thread stages of a K-tile: LOADS float4s of either operand, at a stride from one
    // another, and the next K-tile's at another (no multiplication inside the loop).
    const int64_t step = static_cast<int64_t>(q.share * G) * BK;
    int64_t k0 = static_cast<int64_t>(rank * G + group) * BK;
    constexpr int QUADS = TILE / 4, SPREAD = GROUP / QUADS;  // a row of the tile by k in float4s; k's that a load covers
    struct Side {
        const float* at;
        int64_t between, ahead;
        bool there[LOADS];
        int k;  // of the first load, behind k0
    } sa, sb;
    auto side = [&](const float* base, bool by_k, int64_t first, int64_t extent) {
        Side s;
        s.k = by_k ? tid / QUADS : tid % 2 * 4;
        const int64_t row = first + (by_k ? tid % QUADS * 4 : tid / 2);
        s.at = by_k ? base + (k0 + s.k) * extent + row : base + row * q.K + k0 + s.k;
        s.between = by_k ? SPREAD * extent : GROUP / 2 * q.K;
        s.ahead = by_k ? step * extent : step;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) s.there[l] = row + (by_k ? 0 : l * (GROUP / 2)) < extent;
        return s;
    };
    sa = side(q.A, A_KM, m0, q.M), sb = side(q.B, !B_NK, n0, q.N);
    float4 ra[LOADS], rb[LOADS];
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load = [&](int64_t k) {  // K-tile k, then on to the next
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            ra[l] = sa.there[l] && k + sa.k + (A_KM ? l * SPREAD : 0) < q.K ? *reinterpret_cast<const float4*>(sa.at + l * sa.between) : zero;
            rb[l] = sb.there[l] && k + sb.k + (B_NK ? 0 : l * SPREAD) < q.K ? *reinterpret_cast<const float4*>(sb.at + l * sb.between) : zero;
        }
        sa.at += sa.ahead, sb.at += sb.ahead;
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
    auto of_block = [&](int at) {  // four values, the warps' sums in order
        float4 o = *reinterpret_cast<const float4*>(smem + at);
#pragma unroll
        for (int k = 1; k < G; ++k) add(o, *reinterpret_cast<const float4*>(smem + k * TILE * TILE + at));
        return o;
    };
    int e0 = 0, e1 = TILE * TILE / 4;  // the float4s that this block finishes
    if (q.share > 1) {
        for (int e = static_cast<int>(threadIdx.x); e < e1; e += G * GROUP) *reinterpret_cast<float4*>(smem + 4 * e) = of_block(4 * e);
        if (sums && threadIdx.x < TILE) {
            float t = colsums[threadIdx.x];
#pragma unroll
            for (int k = 1; k < G; ++k) t += colsums[k * TILE + threadIdx.x];
            colsums[threadIdx.x] = t;
        }
        ptx::cluster_sync();
        e1 /= q.share, e0 = rank * e1, e1 += e0;
    }
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += G * GROUP) {
        const int row = e / (TILE / 4), col = e % (TILE / 4) * 4;
        const int64_t m = m0 + row, n = n0 + col;
        if (m >= q.M || n >= q.N) continue;  // N is a multiple of 4: a float4 is all in or all out
        float4 o;
        if (q.share > 1) {
            o = ld_cluster(smem + 4 * e, 0);
            for (int r = 1; r < q.share; ++r) add(o, ld_cluster(smem + 4 * e, r));
        } else {
            o = of_block(4 * e);
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
        if (EPI == DPRE && p.pre) {
            const float4 x = *reinterpret_cast<const float4*>(p.pre + at);
            act::with(p.act, [&](auto kind) {
                constexpr int ACT = decltype(kind)::value;
                o.x *= act::slope<ACT>(x.x), o.y *= act::slope<ACT>(x.y);
                o.z *= act::slope<ACT>(x.z), o.w *= act::slope<ACT>(x.w);
            });
        }
        *reinterpret_cast<float4*>(q.D + at) = o;
    }
    if (sums && q.share == 1 && threadIdx.x < TILE && m0 + threadIdx.x < q.M) {
        float s = colsums[threadIdx.x];
#pragma unroll
        for (int k = 1; k < G; ++k) s += colsums[k * TILE + threadIdx.x];
        p.dbias[m0 + threadIdx.x] = s;
    }
    if (q.share > 1) {
        if (sums && rank == 0 && threadIdx.x < TILE / 4 && m0 + 4 * threadIdx.x < q.M) {  // (M is a multiple of 4 there)
            float4 s = ld_cluster(colsums + 4 * threadIdx.x, 0);
            for (int r = 1; r < q.share; ++r) add(s, ld_cluster(colsums + 4 * threadIdx.x, r));
            *reinterpret_cast<float4*>(p.dbias + m0 + 4 * threadIdx.x) = s;
        }
        ptx::cluster_sync();  // a block's sums stay until the others have read them
    }
}

// Tile and rank of block `b` of a product's blocks; the rank where K is not shared: 0.
__device__ __forceinline__ int tile_of(const Product& q, int b, int& rank) {
    rank = b % q.share;
    return b / q.share;
}

template <int TM, int G>
__global__ void __launch_bounds__(G* GROUP, TM == 4 ? 2 : 1) small_forward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    int rank;
    const int tile = tile_of(p.first, static_cast<int>(blockIdx.x), rank);
    tile_product<TM, G, false, true, FORWARD>(p, p.first, tile, rank, smem);
}

template <int TM, int G>
__global__ void __launch_bounds__(G* GROUP, TM == 4 ? 2 : 1) small_backward_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float smem[];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    // the tiles with the longer sums first: the others fill the gaps behind them
    int b = static_cast<int>(blockIdx.x), rank;
    const bool first_first = p.first.K >= p.second.K;
    const int ahead = first_first ? p.first.blocks(p.cluster) : p.second.blocks(p.cluster);
    const bool dweight = first_first == (b < ahead);
    if (b >= ahead) b -= ahead;
    const int tile = tile_of(dweight ? p.first : p.second, b, rank);
    if (tile >= (dweight ? p.first.tiles : p.second.tiles)) return;  // (fills a cluster that shares nothing)
    if (dweight) tile_product<TM, G, true, false, DWEIGHT>(p, p.first, tile, rank, smem);
    else tile_product<TM, G, false, false, DPRE>(p, p.second, tile, rank, smem);
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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

int64_t tiles_of(int64_t M, int64_t N, int tile) { return (M + tile - 1) / tile * ((N + tile - 1) / tile); }

Product product(float* D, const float* A, const float* B, int64_t M, int64_t N, int64_t K, int tile) {
    return {D, A, B, M, N, K, static_cast<int>((N + tile - 1) / tile), static_cast<int>(tiles_of(M, N, tile))};
}

}  // namespace

namespace {

// Blocks of a cluster that share the K of a product's tiles, a power of two: as many as have
// an SM each, with a K-tile at least for every warp; of tiles of 32 half an SM each where K is long (18 x
// 3732 -> 4032 70 -> 40 us, 100 x 768 -> 768 16.4 -> 12.5, but of shorter ones 200 x 264 -> 388's
// gradients 8.2 -> 11.5, 40 x 600 -> 600 7.3 -> 10.1). Of two products the one that wants more is
// shared, or both.
int share_products(Product* q, int n, int tile, int num_sms) {
    int cluster = 1;
    for (int i = 0; i < n; ++i) {
        const int64_t tiles = tiles_of(q[i].M, q[i].N, tile);
        q[i].share = 1;
        auto room = [&](int share) { return tile == 32 && q[i].K >= 384 * share ? 2 * num_sms : num_sms; };
        while (q[i].share < 8 && 2 * q[i].share * tiles <= room(2 * q[i].share) && 2 * q[i].share * 64 <= q[i].K) q[i].share *= 2;
        cluster = std::max(cluster, q[i].share);
    }
    for (int i = 0; i < n; ++i)
        if (q[i].share < cluster) q[i].share = 1;
    return cluster;
}

// Time models (us), fitted to the measurements below; times (us) on one GB300:
//                         tokens  32 x 32  64 x 64  spans (forward | backward 32, 64, spans)
//     6 x   92 -> 2072         3.6      3.5      5.8   11.7 |  7.4 12.2 53.6
//    16 x 6400 -> 1600        28.9     38.2     55.5    148 |  108  127 58.7
//    18 x 3732 -> 4032                 39.8     56.2   94.4 |  156  195  105
//    40 x  600 ->  600         7.6      7.4      8.6   23.6 |  8.9 14.3 22.3
//    40 x 1600 -> 6400                 63.5     51.2   46.9 |  127  148  154
//    64 x 4000 ->   64         5.8      9.6     18.7   95.4 |  7.2  7.7 13.0
//   100 x  768 ->  768                 12.5     10.7   27.2 | 14.9 17.6 26.4
//   100 x  768 -> 2304                 19.4     16.0   27.4 | 33.9 34.8 61.2
//   200 x  264 ->  388                  7.4      7.7   17.6 |  8.2 10.3 19.1
//   333 x  772 -> 1300                 27.2     24.4   28.6 | 46.5 44.9 39.1
//   407 x 1120 ->  408                 26.5     20.8   35.8 | 26.2 28.0 21.2
//   500 x  768 ->  768                 27.7     24.5   28.1 | 38.6 36.9 27.7
//  1000 x 1600 -> 1600                  185      130   47.5 |  285  227 79.8
//  2048 x 1600 -> 2400                  530      346   88.3 |  819  631  259
// A block of 32 x 32 outputs takes 0.0148 us per value of K alone on its SM and 0.0107 beside
// others, and as long as 60 values more for its first loads and its sums; one of 64 x 64
// 0.0265 and 0.0298, and 120 values more; below 64 values some warps have none. Blocks that
// share a tile take 1.5 to join (64 x 4000 -> 64 in tiles of 32 41 us alone, 9.6 shared by eight). The tensor
// cores' items of 256 x 128 take 0.72 us a k-block of 32 and 4 for the epilogue, 7 for the
// launch and its first loads.
double small_us(int tile, const Product* q, int n, int num_sms) {
    Product shared[2] = {q[0], q[n - 1]};
    share_products(shared, n, tile, num_sms);
    double work = 0.0, longest = 0.0;
    for (int i = 0; i < n; ++i) {
        const int share = shared[i].share;
        const double K = static_cast<double>(q[i].K) / share, blocks = static_cast<double>(tiles_of(q[i].M, q[i].N, tile) * share);
        work += blocks * (tile == 32 ? (std::max(K, 64.0) + 60.0) * 0.0107 : (std::max(K, 64.0) + 120.0) * 0.0298);
        const double beside = share > 1 ? std::max(1.0, blocks / num_sms) : 1.0;  // shared tiles: blocks of one SM
        longest = std::max(longest, K * beside * (tile == 32 ? 0.0148 : 0.0265) + (share > 1 ? 1.5 : 0.0));
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
                                      int act, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Params p{product(out, inp, weight, BT, OC, C, tile), {}, bias, residual, pre, nullptr, act, 1};
    p.cluster = share_products(&p.first, 1, tile, num_sms);
    const int blocks = p.first.blocks(p.cluster);
    if (tile == 64) return launch<small_forward_kernel<8, 8>>(p, blocks, 8 * GROUP, smem_bytes<8, 8>(), stream);
    return launch<small_forward_kernel<4, 8>>(p, blocks, 8 * GROUP, smem_bytes<4, 8>(), stream);
}

cudaError_t simt_small_run_launch(int tile, float* dpre, float* dweight, float* dbias, const float* dout,
                                  const float* inp, const float* weight, const float* pre, int64_t BT, int64_t C,
                                  int64_t OC, int act, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Params p{product(dweight, dout, inp, OC, C, BT, tile), product(dpre, dout, weight, BT, C, OC, tile), nullptr, nullptr,
             const_cast<float*>(pre), dbias, act, 1};
    Product q[2] = {p.first, p.second};
    p.cluster = share_products(q, 2, tile, num_sms);
    p.first = q[0], p.second = q[1];
    const int blocks = p.first.blocks(p.cluster) + p.second.blocks(p.cluster);
    if (tile == 64) return launch<small_backward_kernel<8, 8>>(p, blocks, 8 * GROUP, smem_bytes<8, 8>(), stream);
    return launch<small_backward_kernel<4, 8>>(p, blocks, 8 * GROUP, smem_bytes<4, 8>(), stream);
}

}  // namespace mmbwd
