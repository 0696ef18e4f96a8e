// Products of matrices in 8-bit form (include/q8_linear.h) on the sm_103a tensor
// cores: D (M x N) = A (M x K) . B (N x K)^T, with one power-of-two scale per row
// and block of 128 along K.
//
// The block scales go through the tensor core itself: tcgen05.mma of
// kind::mxf8f6f4 multiplies each step of 32 products by both rows' ue8m0 scales
// on its way into the fp32 accumulator, so a block scale costs no pass over the
// accumulator. An MMA takes one byte per row out of a 32-bit scale word in tensor
// memory, and the scales are stored as those words (tiles of 128 rows x 4
// blocks): one tcgen05.cp per 128 rows serves 512 values of K, and the
// instruction descriptor picks the block's byte.
//
// CTA pairs, as in the bf16 kernel: a cluster of two CTAs computes a 256 x bn tile
// (bn 256 or 128) with pair MMAs (M = 256, K = 32); CTA r stages rows
// [128 r, 128 r + 128) of A, its half of the columns of B, the scales of its 128
// rows of A, and the scales of all bn columns. Both operands are K-major; a stage
// is 128 bytes of K per row (128-byte swizzle), which moves as many bytes per
// tensor-core cycle as a bf16 stage (half the bytes, twice the rate).
//
// Tensor memory (512 columns): two accumulators of 256 columns overlap in 64,
// [0, 256) and [192, 448), and leave 64 columns for the scales. The epilogue
// reads the shared columns first and then lets the next tile's MMAs start, so only
// the first chunk of each epilogue is exposed.
//
// Warp roles (10 warps per CTA): 0 TMA producer; 1 MMA issuer (even CTA) or
// forwarder of "stage full" to the even CTA (odd CTA); 2-9 epilogue, two warps per
// tensor-memory lane quadrant, each taking every other 32-column chunk of its 32
// rows: accumulator (+ bias, or old values requested two chunks ahead) rounded once
// and stored from registers, 32 bytes of a row per thread and store.
//
// Work list: the tiles of one or two products (dinp and dweight), each product's
// reduction cut into `splits` ranges of blocks where its tiles alone do not
// fill the pairs; items go to pairs longest first on the host. Partial tiles of
// a cut product are fp32, in the caller's workspace, and a second kernel adds
// them in split order, so no result depends on timing.
//
// Measured (device time in short runs, 2070 MHz): 8192 tokens 1600 -> 6400 59 us (2.9
// PFLOP/s), 6400 -> 1600 54 us (3.1), 768 -> 50304 246 us (2.6); backward of the first, both
// products, 111 us (3.0). Held for seconds the power cap takes a tenth: 65, 61 and 126 us
// for the first, second and last. A k-block (128 of K) of a 256-wide tile takes 0.33 us, which is the round trip
// of six 32 KB stages; a tile's hand-over about 0.5.
//
// Every wait is bounded (q8_wait_limit_ns): one that gives up records the failure in the
// device status word and all roles unwind.
#include "../../include/q8_linear.h"
#include "internal.h"
#include "ops.h"
#include "q8.cuh"
#include "q8.h"

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

namespace mmbwd {

__device__ unsigned int g_q8_status[4];

namespace {

constexpr int BM = 128, PAIR_M = 256;
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * 128, B_BYTES = 128 * 128;
constexpr int SF_BYTES = 3 * 512;  // scales of 128 rows of A and up to 256 of B, four blocks of K
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8, FIRST_EPI = 2;
constexpr int THREADS = 32 * (FIRST_EPI + EPI_WARPS);
constexpr uint32_t TMEM_COLS = 512, ACC1 = 192, SF_COL = 448, SF_STRIDE = 12;
// Scale buffers in tensor memory: a copy into a buffer may only be issued once the
// MMAs of the group of blocks that used it are done. Those of earlier items are
// (an item starts after the one before it has been read out). Within an item, a
// first group of f <= 4 blocks and then groups of four: the copy of group g + SF_BUFS
// at block f + 4 (g + SF_BUFS - 1) follows the refill of its stage, which waited
// for the MMAs up to STAGES blocks before it, and group g ends at block f + 4 g - 1.
constexpr int SF_BUFS = 4;
static_assert(STAGES <= 4 * SF_BUFS - 3 && SF_BUFS * SF_STRIDE <= 64, "scale buffers");

constexpr int BAR_FULL = 0, BAR_EMPTY = STAGES, BAR_ACC_FULL = 2 * STAGES, BAR_ACC_FREE = 2 * STAGES + 1,
              BAR_TEARDOWN = 2 * STAGES + 2, N_BARS = 2 * STAGES + 3;
constexpr int OFF_SF = STAGES * STAGE_BYTES;
constexpr int OFF_BIAS = OFF_SF + STAGES * SF_BYTES;  // the bias of each epilogue warp's columns, fp32, in its order of chunks
constexpr int OFF_BARS = OFF_BIAS + EPI_WARPS * 128 * 4;
constexpr int OFF_MISC = OFF_BARS + N_BARS * 8;  // [0] tensor-memory base, [1] abort flag
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

constexpr int MAX_PAIRS = 128, MAX_ITEMS = 3000;

struct Schedule {
    uint16_t start[MAX_PAIRS + 1];
    uint16_t items[MAX_ITEMS];
};

struct Prod {
    const uint8_t *a_scale, *b_scale;
    const void* bias;
    void* D;
    float* partials;
    int64_t M, N;
    int groups;  // of four blocks, per row of the scales
    int bn, tiles_m, tiles_n, kb, splits, kb_per_split, item0;
    int f32, add;
    int wide;  // rows of D start on multiples of 32 bytes (2), 16 (1), 8 (0)
    uint32_t idesc;
};

struct Params {
    Prod prod[2];
    int n_items, n_prod, table;
    unsigned long long wait_ns;  // limit of a wait
};

struct Maps {
    CUtensorMap a[2], b[2];
};

struct Item {
    int which, pm, n_tile, split, kb0, kb1;
};

__device__ __forceinline__ Item decode(const Params& p, int w) {
    Item it;
    it.which = p.n_prod == 2 && w >= p.prod[1].item0 ? 1 : 0;
    const Prod& d = p.prod[it.which];
    const int local = w - d.item0, rest = local / d.tiles_n;
    it.n_tile = local % d.tiles_n;
    it.pm = rest % d.tiles_m;
    it.split = rest / d.tiles_m;
    it.kb0 = it.split * d.kb_per_split;
    it.kb1 = min(it.kb0 + d.kb_per_split, d.kb);
    return it;
}

__device__ __forceinline__ int item_at(const Params& p, const Schedule& s, int round) {
    const int c = static_cast<int>(blockIdx.x) / 2;
    if (p.table) {
        const int i = s.start[c] + round;
        return i < s.start[c + 1] ? static_cast<int>(s.items[i]) : p.n_items;
    }
    return round * (static_cast<int>(gridDim.x) / 2) + c;
}

__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(THREADS, 1)
    q8_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p,
                   const __grid_constant__ Schedule sch) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem_raw + (base - raw) + OFF_MISC);
    const uint32_t bars = base + OFF_BARS;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(bars + 8u * (BAR_FULL + s), leader ? 2u : 1u);  // own producer, even CTA: and the forwarder
            ptx::mbar_init(bars + 8u * (BAR_EMPTY + s), 1u);
        }
        ptx::mbar_init(bars + 8u * BAR_ACC_FULL, 1u);
        ptx::mbar_init(bars + 8u * BAR_ACC_FREE, 2u * EPI_WARPS);
        ptx::mbar_init(bars + 8u * BAR_TEARDOWN, 1u);
        misc[1] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(base + OFF_MISC, TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    // The launch before this one may still run. The producer waits for it just ahead
    // of its first load, so that its set-up overlaps; all others here: the epilogue
    // touches global memory, and the MMA issuer's and forwarder's first wait would
    // count the other launch's time against its limit.
    if (warp != 0) ptx::grid_dependency_wait();
    const uint32_t tmem = misc[0];
    const q8::Waiter wt{misc + 1, g_q8_status, p.wait_ns};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            for (int i = 0; i < p.n_prod; ++i) {
                ptx::prefetch_tmap(&maps.a[i]);
                ptx::prefetch_tmap(&maps.b[i]);
            }
            uint32_t stage = 0, phase = 0, issued = 0, last_parity = 0;
            bool ok = true, waited = false;
            for (int r = 0; ok; ++r) {
                const int w = item_at(p, sch, r);
                if (w >= p.n_items) break;
                const Item it = decode(p, w);
                const Prod& d = p.prod[it.which];
                const int row0 = it.pm * PAIR_M + static_cast<int>(rank) * BM;
                const int half = d.bn / 2;
                const int n0 = it.n_tile * d.bn, col0 = n0 + static_cast<int>(rank) * half;
                // boxes and scale tiles wholly outside the matrix are not loaded: they
                // would only reach rows and columns of D that are not stored
                const bool has_a = row0 < d.M, has_b = col0 < d.N;
                const int sf_b = d.bn > 128 && n0 + 128 < d.N ? 2 : 1;
                const uint32_t bytes = (has_a ? A_BYTES : 0u) + (has_b ? static_cast<uint32_t>(half) * 128u : 0u);
                const uint32_t sf_bytes = (has_a ? 512u : 0u) + 512u * sf_b;
                const int64_t gstride = static_cast<int64_t>(d.groups) * 512;
                const uint8_t* sa = d.a_scale + (row0 / 128) * gstride;
                const uint8_t* sb = d.b_scale + (n0 / 128) * gstride;
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!wt.wait(bars + 8u * (BAR_EMPTY + stage), phase ^ 1u, q8::SITE_EMPTY, w)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = base + stage * STAGE_BYTES, fb = bars + 8u * (BAR_FULL + stage);
                    const bool sf = kb == it.kb0 || (kb & 3) == 0;
                    ptx::mbar_arrive_expect_tx(fb, bytes + (sf ? sf_bytes : 0u));
                    if (!waited) {
                        ptx::grid_dependency_wait();
                        waited = true;
                    }
                    if (sf) {
                        const uint32_t st = base + OFF_SF + stage * SF_BYTES;
                        const int64_t g = static_cast<int64_t>(kb >> 2) * 512;
                        if (has_a) q8::bulk_load(st, sa + g, 512u, fb);
                        for (int j = 0; j < sf_b; ++j) q8::bulk_load(st + 512u * (1 + j), sb + j * gstride + g, 512u, fb);
                    }
                    if (has_a) ptx::tma_load_2d(at, &maps.a[it.which], fb, kb * 128, row0);
                    if (has_b) ptx::tma_load_2d(at + A_BYTES, &maps.b[it.which], fb, kb * 128, col0);
                    issued |= 1u << stage;
                    last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
            for (int s = 0; s < STAGES; ++s)
                if ((issued >> s) & 1u)
                    wt.wait(bars + 8u * (BAR_FULL + s), (last_parity >> s) & 1u, q8::SITE_TEARDOWN, -1, true);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && lane == 0) {
            // -------------------------------------------------------- MMA issuer
            uint32_t stage = 0, phase = 0, tile = 0, sf_buf = 0;
            bool ok = true;
            for (int r = 0; ok; ++r, ++tile) {
                const int w = item_at(p, sch, r);
                if (w >= p.n_items) break;
                const Item it = decode(p, w);
                const Prod& d = p.prod[it.which];
                // both CTAs' epilogues have read the columns this tile shares with
                // the one before (and, before that, all of this accumulator)
                if (tile > 0 && !wt.wait(bars + 8u * BAR_ACC_FREE, (tile - 1) & 1u, q8::SITE_ACC_FREE, w)) break;
                ptx::tc_fence_after();
                const uint32_t acc = tmem + (tile & 1u) * ACC1;
                uint32_t sfa = 0;
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!wt.wait(bars + 8u * (BAR_FULL + stage), phase, q8::SITE_FULL, w)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (kb == it.kb0 || (kb & 3) == 0) {
                        const uint64_t sd = q8::scale_desc(base + OFF_SF + stage * SF_BYTES);
                        sfa = tmem + SF_COL + sf_buf * SF_STRIDE;
                        if (++sf_buf == SF_BUFS) sf_buf = 0;
                        q8::copy_scales_pair(sfa, sd);
                        q8::copy_scales_pair(sfa + 4, sd + 32);
                        if (d.bn > 128) q8::copy_scales_pair(sfa + 8, sd + 64);
                    }
                    const uint32_t at = base + stage * STAGE_BYTES;
                    const uint64_t a0 = ptx::smem_desc_sw128(at, 16, 1024);
                    const uint64_t b0 = ptx::smem_desc_sw128(at + A_BYTES, 16, 1024);
                    const uint32_t idesc = d.idesc | q8::scale_id(static_cast<uint32_t>(kb) & 3u);
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 values of K: 32 bytes further into each swizzled row
                        q8::mma_mxf8_pair(acc, a0 + 2u * k, b0 + 2u * k, idesc, sfa, sfa + 4, (kb > it.kb0 || k > 0) ? 1u : 0u);
                    ptx::mma_commit_pair_multicast(bars + 8u * (BAR_EMPTY + stage), 0x3u);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                ptx::mma_commit_pair_multicast(bars + 8u * BAR_ACC_FULL, 0x3u);
            }
            ptx::mma_commit_pair(bars + 8u * BAR_TEARDOWN);
            wt.wait(bars + 8u * BAR_TEARDOWN, 0u, q8::SITE_TEARDOWN, -1, true);
        } else if (!leader && lane == 0) {
            // ---------------------------------------------- forwarder (odd CTA)
            const uint32_t full0 = ptx::mapa(bars + 8u * BAR_FULL, 0);
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int w = item_at(p, sch, r);
                if (w >= p.n_items) break;
                const Item it = decode(p, w);
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!wt.wait(bars + 8u * (BAR_FULL + stage), phase, q8::SITE_FORWARD, w)) {
                        ok = false;
                        break;
                    }
                    ptx::mbar_arrive_cluster_relaxed(full0 + 8u * stage);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;                  // tensor-memory lane quadrant this warp may read
        const int h = (warp - FIRST_EPI) >> 2;   // which of the quadrant's two warps
        const uint32_t free_bar = ptx::mapa(bars + 8u * BAR_ACC_FREE, 0);
        // 32-column chunk that this warp takes in step k of its t-th tile: the shared
        // columns (the last 64 of the even accumulator, the first 64 of the odd one) first
        auto chunk_of = [&](int bn, uint32_t t, int k) {
            return (bn == 256 && (t & 1u) == 0) ? (k == 0 ? 6 + h : 2 * (k - 1) + h) : 2 * k + h;
        };
        // The bias of the columns of tile r, one a lane and step: requested a tile
        // ahead and then kept in shared memory, where all lanes read the same value
        // (the L1 that the stages leave loses it to the stores: loads in the epilogue
        // took 4096 tokens 768 -> 50304 from 122 us without a bias to 226, and 350 with
        // an fp32 output; this way 150 and 222).
        float* const bias_s = reinterpret_cast<float*>(smem_raw + (base - raw) + OFF_BIAS) + (warp - FIRST_EPI) * 128;
        uint32_t bias_r[4] = {0u, 0u, 0u, 0u};  // as loaded: converting here would wait for the load
        const Prod& only = p.prod[0];           // (two products in one launch have no bias)
        auto fetch_bias = [&](int r) {
            const int w = only.bias ? item_at(p, sch, r) : p.n_items;
            if (w >= p.n_items) return;
            const int first = w % only.tiles_n * only.bn;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = first + chunk_of(only.bn, static_cast<uint32_t>(r), k) * 32 + lane, at = c < only.N ? c : only.N - 1;
                bias_r[k] = only.f32 ? static_cast<const uint32_t*>(only.bias)[at] : static_cast<const uint16_t*>(only.bias)[at];
            }
        };
        fetch_bias(0);
        uint32_t tile = 0;
        for (int r = 0;; ++r, ++tile) {
            const int w = item_at(p, sch, r);
            if (w >= p.n_items) break;
            const Item it = decode(p, w);
            const Prod& d = p.prod[it.which];
            const int64_t row = static_cast<int64_t>(it.pm) * PAIR_M + static_cast<int>(rank) * BM + q * 32 + lane;
            const int col0 = it.n_tile * d.bn;
            const int nk = d.bn / 64;  // this warp's 32-column chunks of the tile
            const bool in_row = row < d.M;
            auto chunk = [&](int k) { return chunk_of(d.bn, tile, k); };
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (tile & 1u) * ACC1;
            auto release = [&](int k) {  // after the first chunk has been read
                if (k > 0) return;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(free_bar);
            };
            if (d.bias) {
                __syncwarp();  // the tile before has read its own
#pragma unroll
                for (int k = 0; k < 4; ++k) bias_s[32 * k + lane] = __uint_as_float(d.f32 ? bias_r[k] : bias_r[k] << 16);
                __syncwarp();
                fetch_bias(r + 1);
            }
            auto add_bias = [&](int k, uint32_t (&v)[32]) {
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const float4 b = reinterpret_cast<const float4*>(bias_s + 32 * k)[g];
                    v[4 * g] = __float_as_uint(__uint_as_float(v[4 * g]) + b.x);
                    v[4 * g + 1] = __float_as_uint(__uint_as_float(v[4 * g + 1]) + b.y);
                    v[4 * g + 2] = __float_as_uint(__uint_as_float(v[4 * g + 2]) + b.z);
                    v[4 * g + 3] = __float_as_uint(__uint_as_float(v[4 * g + 3]) + b.w);
                }
            };
            if (d.splits > 1) {  // partial sums: [128-row tile x column tile][split][128][bn]
                if (!wt.wait_warp(bars + 8u * BAR_ACC_FULL, tile & 1u, q8::SITE_ACC_FULL, w)) break;
                ptx::tc_fence_after();
                float* dst = d.partials +
                             (((static_cast<int64_t>(it.pm * 2 + static_cast<int>(rank)) * d.tiles_n + it.n_tile) * d.splits + it.split) * BM +
                              q * 32 + lane) * d.bn;
#pragma unroll 1
                for (int k = 0; k < nk; ++k) {
                    uint32_t v[32];
                    const int c = chunk(k) * 32;
                    ptx::tmem_ld32(acc + c, v);
                    release(k);
                    if (in_row) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) q8::st256(dst + c + 8 * g, v + 8 * g);
                    }
                }
            } else if (d.f32) {
                float* D = static_cast<float*>(d.D) + row * d.N + col0;
                auto store = [&](int c, const uint32_t (&v)[32]) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) q8::st256(D + c + 8 * g, v + 8 * g, in_row ? d.N - col0 - c - 8 * g : 0, 4, d.wide);
                };
                if (d.add) {  // the old values two chunks ahead
                    uint32_t old[2][32];
                    auto fetch = [&](int k) {
                        const int c = chunk(k) * 32;
#pragma unroll
                        for (int g = 0; g < 4; ++g) q8::ld256(D + c + 8 * g, old[k & 1] + 8 * g, in_row ? d.N - col0 - c - 8 * g : 0, 4, d.wide);
                    };
                    fetch(0), fetch(1);
                    if (!wt.wait_warp(bars + 8u * BAR_ACC_FULL, tile & 1u, q8::SITE_ACC_FULL, w)) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= nk) break;
                        uint32_t v[32];
                        const int c = chunk(k) * 32;
                        ptx::tmem_ld32(acc + c, v);
                        release(k);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(old[k & 1][e]));
                        if (k + 2 < nk) fetch(k + 2);
                        store(c, v);
                    }
                } else {
                    if (!wt.wait_warp(bars + 8u * BAR_ACC_FULL, tile & 1u, q8::SITE_ACC_FULL, w)) break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < nk; ++k) {
                        uint32_t v[32];
                        const int c = chunk(k) * 32;
                        ptx::tmem_ld32(acc + c, v);
                        release(k);
                        if (d.bias) add_bias(k, v);
                        store(c, v);
                    }
                }
            } else {
                __nv_bfloat16* D = static_cast<__nv_bfloat16*>(d.D) + row * d.N + col0;
                auto store = [&](int c, const uint32_t (&o)[16]) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) q8::st256(D + c + 16 * g, o + 8 * g, in_row ? d.N - col0 - c - 16 * g : 0, 8, d.wide);
                };
                if (d.add) {
                    uint32_t old[2][16];
                    auto fetch = [&](int k) {
                        const int c = chunk(k) * 32;
#pragma unroll
                        for (int g = 0; g < 2; ++g) q8::ld256(D + c + 16 * g, old[k & 1] + 8 * g, in_row ? d.N - col0 - c - 16 * g : 0, 8, d.wide);
                    };
                    fetch(0), fetch(1);
                    if (!wt.wait_warp(bars + 8u * BAR_ACC_FULL, tile & 1u, q8::SITE_ACC_FULL, w)) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= nk) break;
                        uint32_t v[32], o[16];
                        const int c = chunk(k) * 32;
                        ptx::tmem_ld32(acc + c, v);
                        release(k);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = pack_bf16(__uint_as_float(v[2 * e]) + lo_bf16(old[k & 1][e]),
                                             __uint_as_float(v[2 * e + 1]) + hi_bf16(old[k & 1][e]));
                        if (k + 2 < nk) fetch(k + 2);
                        store(c, o);
                    }
                } else {
                    if (!wt.wait_warp(bars + 8u * BAR_ACC_FULL, tile & 1u, q8::SITE_ACC_FULL, w)) break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < nk; ++k) {
                        uint32_t v[32], o[16];
                        const int c = chunk(k) * 32;
                        ptx::tmem_ld32(acc + c, v);
                        release(k);
                        if (d.bias) add_bias(k, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = pack_bf16(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        store(c, o);
                    }
                }
            }
        }
    }

    ptx::grid_launch_dependents();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the even CTA's MMAs use both CTAs' memory
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// D = (old D +) partial_0 + partial_1 + ... in split order, rounded once; four
// columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) q8_join_kernel(T* D, const float* __restrict__ partials, int64_t M, int64_t N,
                                                      int bn, int tiles_n, int splits, int add) {
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t per_row = N / 4, n = M * per_row, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t tile = static_cast<int64_t>(BM) * bn;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
        const int64_t row = i / per_row, col = (i - row * per_row) * 4;
        const float* src = partials + ((row / BM) * tiles_n + col / bn) * splits * tile + (row % BM) * bn + col % bn;
        float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
        if (add) {
            if constexpr (sizeof(T) == 4) {
                old = *reinterpret_cast<const float4*>(D + row * N + col);
            } else {
                const uint2 o = *reinterpret_cast<const uint2*>(D + row * N + col);
                old = make_float4(lo_bf16(o.x), hi_bf16(o.x), lo_bf16(o.y), hi_bf16(o.y));
            }
        }
        float4 s = __ldcg(reinterpret_cast<const float4*>(src));
#pragma unroll 4
        for (int k = 1; k < splits; ++k) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src + k * tile));
            s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
        }
        if (add) s.x += old.x, s.y += old.y, s.z += old.z, s.w += old.w;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(D + row * N + col) = s;
        else
            *reinterpret_cast<uint2*>(D + row * N + col) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

// ------------------------------------------------------------------ planning

struct ProductPlan {
    int bn, tiles_m, tiles_n, kb, splits, kb_per_split, item0, items;
    double epi;  // us of a 256-column epilogue
    size_t ws_off, ws_bytes;
};

struct Plan {
    ProductPlan p[2];
    int n, n_items, table, grid;
    size_t ws_bytes;
    Schedule sched;
};

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Time model (us): a block of K costs t_kb, an item a handoff (the first chunk of
// its epilogue) and, at the end, an epilogue that nothing overlaps; a split
// product the pass that joins its partials.
double kb_us(int bn) { return bn == 256 ? 0.30 : 0.22; }
constexpr double ITEM_US = 0.6;
double epi_us(const ProductPlan& p) { return (p.splits > 1 ? 3.0 : p.epi) * p.bn / 256.0; }

// A 256-column epilogue: plain stores are not waited for, adding to the old values is
// (a dweight of 9728 x 2048 from 8 tokens, four rounds of tiles: fp32 22.1 us, added to
// 38.4; bf16 14.4 and 20.1). Widths and splits are searched with the first cost, so
// that the workspace depends on the shapes alone; items are then assigned to pairs
// by their own (512 tokens, C = 1600, OC = 6400, fp32 dweight added to: 34.2 -> 27.5 us;
// with dearer plain stores too, 2200 x 8680 without adding got slower, 28.7 -> 31.6).
constexpr double EPI_SEARCH = 2.0;
double epi_of(bool f32, bool add) { return !add ? EPI_SEARCH : f32 ? 8.5 : 4.0; }

double item_us(const ProductPlan& p, int split) {
    const int k0 = split * p.kb_per_split, k1 = std::min(k0 + p.kb_per_split, p.kb);
    return std::max((k1 - k0) * kb_us(p.bn), epi_us(p)) + ITEM_US;
}

double join_us(const ProductPlan& p, int64_t M, int64_t N) {
    return p.splits == 1 ? 0.0 : 2.5 + static_cast<double>(M) * N * 4.0 * (p.splits + 1) / 8e6;
}

// Longest item first, each to the pair with the least work (ties to the lower
// pair, items in order): a pure function of the plan. Returns the makespan.
double assign(Plan& pl, int pairs) {
    static thread_local double load[MAX_PAIRS];
    static thread_local int cnt[MAX_PAIRS], order[MAX_ITEMS];
    static thread_local float cost[MAX_ITEMS];
    static thread_local uint8_t owner[MAX_ITEMS];
    for (int i = 0; i < pl.n; ++i) {
        const ProductPlan& p = pl.p[i];
        const int tiles = p.tiles_m * p.tiles_n;
        for (int k = 0; k < p.items; ++k) cost[p.item0 + k] = static_cast<float>(item_us(p, k / tiles));
    }
    for (int w = 0; w < pl.n_items; ++w) order[w] = w;
    std::stable_sort(order, order + pl.n_items, [&](int a, int b) { return cost[a] > cost[b]; });
    for (int c = 0; c < pairs; ++c) load[c] = 0.0, cnt[c] = 0;
    for (int k = 0; k < pl.n_items; ++k) {
        int best = 0;
        for (int c = 1; c < pairs; ++c)
            if (load[c] < load[best] - 1e-9) best = c;
        load[best] += cost[order[k]];
        owner[k] = static_cast<uint8_t>(best);
        ++cnt[best];
    }
    pl.sched.start[0] = 0;
    for (int c = 0; c < MAX_PAIRS; ++c)
        pl.sched.start[c + 1] = static_cast<uint16_t>(pl.sched.start[c] + (c < pairs ? cnt[c] : 0));
    int fill[MAX_PAIRS];
    for (int c = 0; c < pairs; ++c) fill[c] = pl.sched.start[c];
    for (int k = 0; k < pl.n_items; ++k) pl.sched.items[fill[owner[k]]++] = static_cast<uint16_t>(order[k]);
    double m = 0.0;
    for (int c = 0; c < pairs; ++c) m = std::max(m, load[c]);
    return m;
}

// The makespan where pairs take the items in turn (more items than the schedule
// holds): pair c has those of c, c + pairs, ...
double in_turn_us(const Plan& pl, int pairs) {
    double m = 0.0;
    for (int c = 0; c < pairs; ++c) {
        auto before = [&](int w) { return w > c ? (w - c + pairs - 1) / pairs : 0; };  // of this pair's items
        double t = 0.0;
        for (int i = 0; i < pl.n; ++i) {
            const ProductPlan& p = pl.p[i];
            const int tiles = p.tiles_m * p.tiles_n;
            for (int k = 0; k < p.splits; ++k) {
                const int first = p.item0 + k * tiles;
                t += (before(first + tiles) - before(first)) * item_us(p, k);
            }
        }
        m = std::max(m, t);
    }
    return m;
}

struct Shape3 {
    int64_t M, N, K;
};

// Overrides for tuning and tests: MMBWD_Q8_TILE_N and MMBWD_Q8_SPLITS = "<dinp>,<dweight>"
// (0: the planner's choice; the forward's tile width is the first), here in the
// order of a launch's products.
struct Forced {
    int bn[2], splits[2];
};

Forced forced_from_env(const Q8Product* products, int n) {
    Forced f{};
    if (const char* t = std::getenv("MMBWD_Q8_TILE_N")) {
        int a = 0, b = 0;
        if (std::sscanf(t, "%d,%d", &a, &b) == 2) {
            f.bn[0] = a == 128 || a == 256 ? a : 0;
            f.bn[1] = b == 128 || b == 256 ? b : 0;
        }
    }
    if (const char* t = std::getenv("MMBWD_Q8_SPLITS")) {
        int a = 0, b = 0;
        if (std::sscanf(t, "%d,%d", &a, &b) == 2) f.splits[0] = std::max(0, std::min(a, 16)), f.splits[1] = std::max(0, std::min(b, 16));
    }
    if (n == 1) {
        f.bn[0] = f.bn[products[0].slot], f.splits[0] = f.splits[products[0].slot];
        f.bn[1] = f.splits[1] = 0;
    }
    return f;
}

// What a search finds: tile width and split count of each product; bn[0] == 0 where
// no candidate is possible (an override that cuts a product into more items than
// the schedule holds).
struct Choice {
    int bn[2], splits[2];
};

// The plan of a choice, its items not yet assigned to pairs; false where it is
// not possible.
bool lay_out(const Shape3* s, int n, const Choice& ch, int num_sms, Plan* pl) {
    const int max_pairs = std::max(1, std::min(num_sms / 2, MAX_PAIRS));
    pl->n = n;
    pl->n_items = 0;
    pl->ws_bytes = 0;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        ProductPlan& p = pl->p[i];
        p.bn = ch.bn[i];
        p.epi = EPI_SEARCH;
        p.tiles_m = ceil_div(s[i].M, PAIR_M);
        p.tiles_n = ceil_div(s[i].N, p.bn);
        p.kb = ceil_div(s[i].K, 128);
        p.kb_per_split = ceil_div(p.kb, std::min(ch.splits[i], p.kb));
        p.splits = ceil_div(p.kb, p.kb_per_split);
        if (ch.splits[i] > 1 && p.splits != ch.splits[i]) return false;
        const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
        p.item0 = static_cast<int>(total);
        total += tiles * p.splits;
        if (total > INT32_MAX) return false;
        p.items = static_cast<int>(tiles * p.splits);
        p.ws_off = pl->ws_bytes;
        const int64_t part_rows = 2 * tiles * p.splits * BM;
        if (p.splits > 1 && (part_rows > INT32_MAX || p.items > MAX_ITEMS)) return false;  // (bounds the workspace)
        p.ws_bytes = p.splits > 1 ? static_cast<size_t>(part_rows) * p.bn * 4 : 0;
        pl->ws_bytes += p.ws_bytes;
    }
    pl->n_items = static_cast<int>(total);
    pl->table = pl->n_items <= MAX_ITEMS ? 1 : 0;
    pl->grid = 2 * static_cast<int>(std::min<int64_t>(total, max_pairs));
    return true;
}

// The best choice by the time model over tile widths and, where allowed, splits.
Choice search(const Shape3* s, int n, bool may_split, const Forced& force, int num_sms) {
    static thread_local Plan c;
    double best = 1e300;
    Choice found{};
    static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    for (int widths = 0; widths < (n == 2 ? 4 : 2); ++widths)
        for (int s0 : kSplits)
            for (int s1 : kSplits) {
                if ((n == 1 && s1 > 1) || (!may_split && (s0 > 1 || s1 > 1))) continue;
                const Choice ch{{widths & 1 ? 128 : 256, widths & 2 ? 128 : 256}, {s0, s1}};
                bool skip = false;
                for (int i = 0; i < n; ++i) {
                    if (force.bn[i] && force.bn[i] != ch.bn[i]) skip = true;
                    // a forced count above the number of blocks, or one that would leave
                    // an empty range, is lowered to the nearest that does not
                    if (may_split && force.splits[i]) {
                        const int kb = ceil_div(s[i].K, 128), per = ceil_div(kb, std::min(force.splits[i], kb));
                        const int count = ceil_div(kb, per);
                        int usable = 1;
                        for (int o : kSplits)
                            if (o <= count && ceil_div(kb, ceil_div(kb, o)) == o) usable = o;
                        if (ch.splits[i] != usable) skip = true;
                    }
                }
                if (skip || !lay_out(s, n, ch, num_sms, &c)) continue;
                double work = 0.0, longest = 0.0, tail = 0.0;
                for (int i = 0; i < n; ++i) {
                    const ProductPlan& p = c.p[i];
                    for (int k = 0; k < p.splits; ++k) {
                        work += item_us(p, k) * (p.items / p.splits);
                        longest = std::max(longest, item_us(p, k));
                    }
                    tail += join_us(p, s[i].M, s[i].N);
                }
                const int pairs = c.grid / 2;
                if (std::max(work / pairs, longest) + tail >= best) continue;
                const double t = tail + (c.table ? assign(c, pairs) : in_turn_us(c, pairs));
                if (t < best) {
                    best = t;
                    found = ch;
                }
            }
    return found;
}

// Choices and plans are pure functions of their keys, remembered for the last shapes
// seen: the choice by shapes, SM count and overrides; the plan, whose items are
// assigned by what the epilogues store, by that too. Both are made without a lock.
struct Key {
    int64_t v[15];
};

Key make_key(const Shape3* s, int n, bool may_split, const Forced& f, int num_sms) {
    Key k{};
    for (int i = 0; i < n; ++i) k.v[3 * i] = s[i].M, k.v[3 * i + 1] = s[i].N, k.v[3 * i + 2] = s[i].K;
    k.v[6] = n, k.v[7] = may_split ? 1 : 0, k.v[8] = num_sms;
    for (int i = 0; i < 2; ++i) k.v[9 + i] = f.bn[i], k.v[11 + i] = f.splits[i];
    return k;
}

// SETS sets (a power of two) of WAYS entries; the least recently used of a set goes.
template <typename V, int SETS, int WAYS>
struct Cache {
    struct Entry {
        Key key;
        uint64_t used;  // 0: empty
        V value;
    };
    Entry e[SETS][WAYS];
    uint64_t clock;
    std::mutex m;

    Entry* set_of(const Key& k) {
        uint64_t h = 1469598103934665603ull;
        for (int64_t x : k.v) {
            h = (h ^ static_cast<uint64_t>(x)) * 0x9E3779B97F4A7C15ull;
            h ^= h >> 32;
        }
        return e[h & (SETS - 1)];
    }
    bool get(const Key& k, V* out) {
        std::lock_guard<std::mutex> g(m);
        Entry* s = set_of(k);
        for (int i = 0; i < WAYS; ++i)
            if (s[i].used && std::memcmp(&s[i].key, &k, sizeof(k)) == 0) {
                s[i].used = ++clock;
                *out = s[i].value;
                return true;
            }
        return false;
    }
    void put(const Key& k, const V& v) {
        std::lock_guard<std::mutex> g(m);
        Entry* s = set_of(k);
        int at = 0;
        for (int i = 0; i < WAYS; ++i) {
            if (s[i].used && std::memcmp(&s[i].key, &k, sizeof(k)) == 0) return;  // another thread was first
            if (s[i].used < s[at].used) at = i;
        }
        s[at].key = k;
        s[at].value = v;
        s[at].used = ++clock;
    }
};
Cache<Choice, 256, 8> g_choices;
Cache<Plan, 32, 8> g_plans;
std::atomic<long long> g_searches{0};

Choice choice_for(const Shape3* s, int n, bool may_split, const Forced& force, int num_sms, const Key& k) {
    Choice ch;
    if (g_choices.get(k, &ch)) return ch;
    ++g_searches;
    ch = search(s, n, may_split, force, num_sms);
    if (ch.bn[0] == 0) ch = search(s, n, may_split, Forced{}, num_sms);
    g_choices.put(k, ch);
    return ch;
}

// The plan of a launch in `out`; n_items == 0: none is possible.
void plan_for(const Shape3* s, const Q8Product* products, int n, bool may_split, int num_sms, Plan* out) {
    const Forced force = forced_from_env(products, n);
    const Key k = make_key(s, n, may_split, force, num_sms);
    Key with_types = k;
    double epi[2] = {0.0, 0.0};
    for (int i = 0; i < n; ++i) {
        epi[i] = epi_of(products[i].dtype == MMBWD_F32, products[i].add != 0);
        with_types.v[13 + i] = static_cast<int64_t>(epi[i] * 16.0);
    }
    if (g_plans.get(with_types, out)) return;
    const Choice ch = choice_for(s, n, may_split, force, num_sms, k);
    if (ch.bn[0] == 0 || !lay_out(s, n, ch, num_sms, out)) {
        out->n_items = 0;
        return;
    }
    for (int i = 0; i < n; ++i) out->p[i].epi = epi[i];
    if (out->table) assign(*out, out->grid / 2);
    g_plans.put(with_types, *out);
}

// ------------------------------------------------------------------ launch

// An operand's 8-bit values: boxes of 128 bytes of K by `box_rows` rows.
bool encode_2d(CUtensorMap* m, const void* base, uint64_t ld, uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn encode = get_encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[2] = {ld, rows}, strides[1] = {ld};
    const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t set_smem_once() {
    static std::mutex m;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> g(m);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(q8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

cudaError_t launch_pair(const Plan& pl, const Q8Product* prod, uint8_t* ws, cudaStream_t stream) {
    cudaError_t e = set_smem_once();
    if (e != cudaSuccess) return e;
    static thread_local Maps maps;
    Params par{};
    par.n_prod = pl.n;
    par.n_items = pl.n_items;
    par.table = pl.table;
    par.wait_ns = q8_wait_limit_ns();
    for (int i = 0; i < pl.n; ++i) {
        const Q8Product& q = prod[i];
        const ProductPlan& pp = pl.p[i];
        const uint64_t ld = static_cast<uint64_t>(q8_ld(q.K)), m = static_cast<uint64_t>(q.M), n = static_cast<uint64_t>(q.N);
        const bool f32 = q.dtype == MMBWD_F32;
        const bool ok = encode_2d(&maps.a[i], q.A, ld, m, BM) && encode_2d(&maps.b[i], q.B, ld, n, static_cast<uint32_t>(pp.bn / 2));
        if (!ok) return cudaErrorInvalidValue;
        Prod& d = par.prod[i];
        d.a_scale = q.a_scale, d.b_scale = q.b_scale, d.bias = q.bias;
        d.D = q.D, d.partials = reinterpret_cast<float*>(ws + pp.ws_off);
        const uint64_t at = reinterpret_cast<uintptr_t>(q.D) | n * (f32 ? 4 : 2);  // (N is a multiple of 4)
        d.wide = at % 32 == 0 ? 2 : at % 16 == 0 ? 1 : 0;
        d.M = q.M, d.N = q.N;
        d.groups = static_cast<int>(q8_groups(q.K));
        d.bn = pp.bn, d.tiles_m = pp.tiles_m, d.tiles_n = pp.tiles_n, d.kb = pp.kb;
        d.splits = pp.splits, d.kb_per_split = pp.kb_per_split, d.item0 = pp.item0;
        d.f32 = f32 ? 1 : 0, d.add = q.add;
        d.idesc = q8::idesc_mxf8(PAIR_M, pp.bn, q.a_format, q.b_format);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.grid), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, q8_pair_kernel, maps, par, pl.sched);
    for (int i = 0; i < pl.n && e == cudaSuccess; ++i) {
        const ProductPlan& pp = pl.p[i];
        if (pp.splits == 1) continue;
        const Q8Product& q = prod[i];
        cudaLaunchConfig_t jc{};
        jc.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((q.M * (q.N / 4) + 255) / 256, 1216))), 1, 1);
        jc.blockDim = dim3(256, 1, 1);
        jc.stream = stream;
        jc.attrs = attr;
        jc.numAttrs = 1;
        const float* part = reinterpret_cast<const float*>(ws + pp.ws_off);
        e = q.dtype == MMBWD_F32
                ? cudaLaunchKernelEx(&jc, q8_join_kernel<float>, static_cast<float*>(q.D), part, q.M, q.N, pp.bn,
                                     pp.tiles_n, pp.splits, q.add)
                : cudaLaunchKernelEx(&jc, q8_join_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16*>(q.D), part, q.M, q.N,
                                     pp.bn, pp.tiles_n, pp.splits, q.add);
    }
    return e;
}

}  // namespace

size_t q8_products_workspace(const Q8Product* products, int n, int num_sms) {
    Shape3 s[2];
    for (int i = 0; i < n; ++i) s[i] = {products[i].M, products[i].N, products[i].K};
    const Forced force = forced_from_env(products, n);
    const Choice ch = choice_for(s, n, true, force, num_sms, make_key(s, n, true, force, num_sms));
    static thread_local Plan pl;
    return ch.bn[0] != 0 && lay_out(s, n, ch, num_sms, &pl) ? pl.ws_bytes : 0;
}

cudaError_t q8_products_launch(const Q8Product* products, int n, bool may_split, void* ws, size_t ws_bytes, int num_sms,
                               cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Shape3 s[2];
    for (int i = 0; i < n; ++i) s[i] = {products[i].M, products[i].N, products[i].K};
    static thread_local Plan pl;
    plan_for(s, products, n, may_split, num_sms, &pl);
    if (pl.n_items == 0 || pl.ws_bytes > ws_bytes) return cudaErrorInvalidValue;
    return launch_pair(pl, products, static_cast<uint8_t*>(ws), stream);
}

long long q8_plan_searches() { return g_searches.load(); }

__global__ void q8_selftest_kernel(unsigned long long limit_ns) { q8::selftest_wait(g_q8_status, limit_ns); }

cudaError_t q8_selftest_wait(unsigned long long limit_ns) {
    q8_selftest_kernel<<<1, 1>>>(limit_ns);
    return cudaGetLastError();
}

cudaError_t q8_read_status(int* code, int* info3, bool reset) {
    unsigned int h[4] = {0, 0, 0, 0};
    cudaError_t e = cudaMemcpyFromSymbol(h, g_q8_status, sizeof(h));
    if (e != cudaSuccess) return e;
    *code = h[0] ? -static_cast<int>(h[0]) : MMBWD_OK;
    for (int i = 0; i < 3; ++i) info3[i] = static_cast<int>(h[1 + i]);
    if (reset) {
        const unsigned int z[4] = {0, 0, 0, 0};
        e = cudaMemcpyToSymbol(g_q8_status, z, sizeof(z));
    }
    return e;
}

}  // namespace mmbwd
