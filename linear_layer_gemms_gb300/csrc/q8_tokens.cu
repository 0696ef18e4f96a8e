// The 8-bit forward for few tokens (include/q8_linear.h, mmbwd_q8_forward):
// out (T x N) = inp (T x K) . weight (N x K)^T + bias where the weight's bytes are the
// work.
//
// The product is turned around: 128 rows of the weight are the MMA's M side and
// NT tokens (16, 32 or 64) its N side, so a small T does not fill most of a
// 256-row tile with nothing; more tokens are more tiles. Block scales enter the
// MMA as in the pair kernel (q8_product.cu). Two CTAs per SM, each with a ring of up
// to 100 KB. One token 1600 -> 4800 takes 5.2 us (1.5 TB/s of weights), 16 tokens 768 ->
// 50304 9.3 us (4.2 TB/s), 16 tokens 12800 -> 4096 11.7 us (4.5 TB/s).
//
// Tiles alone fill the device when there are many (a vocabulary): CTAs then
// walk them, the loads of the next tile running beside the epilogue of the last
// (two accumulators). When there are few, one SM's loads from HBM are the limit
// (about 50 GB/s measured), so the S CTAs of a cluster (2, 4 or 8, as many as can be
// resident) share a tile's K: each writes its fp32 partial sums of a token into the
// shared memory of the CTA that owns the token, and after one cluster barrier
// the owner adds them in rank order. One launch, no workspace, the same bits on
// every call.
//
// Warps: 0 producer, 1 MMA issuer, 2-5 epilogue (lane = weight row, so that 32
// lanes write neighbouring outputs).
//
// Every wait is bounded (q8_wait_limit_ns) and recorded when it gives up; all threads still
// reach the cluster barriers.
#include "../../include/q8_linear.h"
#include "internal.h"
#include "ops.h"
#include "q8.cuh"
#include "q8.h"

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>

namespace mmbwd {

__device__ unsigned int g_q8_tokens_status[4];

namespace {

constexpr int ROWS = 128;  // weight rows of a tile
constexpr int THREADS = 192;

template <int NT>
struct Cfg {
    static constexpr int STAGE = ROWS * 128 + NT * 128;
    static constexpr int STAGES = NT == 16 ? 5 : NT == 32 ? 4 : 3;
    static constexpr int OFF_PART = STAGES * STAGE;  // partial sums [rank][owned token][128], fp32
    static constexpr int OFF_SF = OFF_PART + NT * ROWS * 4;  // per stage: 512 bytes of the weight's scales, 512 of the tokens'
    static constexpr int OFF_BARS = OFF_SF + STAGES * 1024;
    static constexpr int N_BARS = 2 * STAGES + 5;
    static constexpr int OFF_MISC = OFF_BARS + N_BARS * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    // Scale buffers in tensor memory (8 columns each), rewritten only after the MMAs
    // that read them: within a tile as in q8_product.cu; from tile to tile, a tile of two
    // blocks or more puts four groups at least STAGES blocks apart, and with one block to
    // a tile the wait for the accumulator of two tiles before covers it.
    static constexpr int SF_BUFS = 4;
    static constexpr uint32_t ACC = NT < 32 ? 32 : NT;  // columns between the two accumulators
    static constexpr uint32_t SF_COL = 2 * ACC;
    static constexpr uint32_t TMEM_COLS = NT <= 32 ? 128 : 256;
    static_assert(STAGES <= 4 * SF_BUFS - 3 && STAGES <= 2 * SF_BUFS - 2, "a scale buffer is rewritten only after its MMAs");
    static_assert(SF_COL + 8 * SF_BUFS <= TMEM_COLS, "tensor memory");
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs on an SM");
};

struct Params {
    void* out;
    const void* bias;
    const uint8_t *w_scale, *x_scale;
    int64_t T, N;
    int64_t groups;
    int kb, tiles, tiles_n, splits, f32;
    uint32_t idesc;
    unsigned long long wait_ns;  // limit of a wait
};

template <int NT>
__global__ void __launch_bounds__(THREADS, 2)
    q8_tokens_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ Params p) {
    using L = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem_raw + (base - raw) + L::OFF_MISC);
    const uint32_t full = base + L::OFF_BARS, empty = full + 8u * L::STAGES;
    const uint32_t acc_full = empty + 8u * L::STAGES, acc_free = acc_full + 16u;  // two of each
    const uint32_t teardown = acc_free + 16u;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    // splits > 1: one tile per cluster; else the CTA's tiles are first, first + step, ...
    const int rank = static_cast<int>(blockIdx.x) % p.splits, first = static_cast<int>(blockIdx.x) / p.splits;
    const int step = static_cast<int>(gridDim.x) / p.splits;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / p.splits);  // > kb0: splits <= kb

    if (threadIdx.x == 0) {
        ptx::prefetch_tmap(&tm_w);
        ptx::prefetch_tmap(&tm_x);
        for (int s = 0; s < L::STAGES; ++s) {
            ptx::mbar_init(full + 8u * s, 1u);
            ptx::mbar_init(empty + 8u * s, 1u);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(acc_full + 8u * i, 1u);
            ptx::mbar_init(acc_free + 8u * i, 4u);
        }
        ptx::mbar_init(teardown, 1u);
        misc[1] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + L::OFF_MISC, L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (p.splits > 1) ptx::cluster_sync();  // the ranks' shared memory exists before it is written
    ptx::tc_fence_after();
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const uint32_t tmem = misc[0];
    const q8::Waiter wt{misc + 1, g_q8_tokens_status, p.wait_ns};
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0, last_parity = 0;
            for (int tile = first; tile < p.tiles && ok; tile += step) {
                const int n0 = tile % p.tiles_n * ROWS;
                const int64_t t0 = static_cast<int64_t>(tile / p.tiles_n) * NT;
                const uint8_t* sw = p.w_scale + (n0 / 128) * p.groups * 512;
                const uint8_t* sx = p.x_scale + (t0 / 128) * p.groups * 512;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wt.wait(empty + 8u * stage, phase ^ 1u, q8::SITE_EMPTY, tile)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = base + stage * L::STAGE, bar = full + 8u * stage;
                    const bool sf = kb == kb0 || (kb & 3) == 0;
                    ptx::mbar_arrive_expect_tx(bar, L::STAGE + (sf ? 1024u : 0u));
                    ptx::tma_load_2d(at, &tm_w, bar, kb * 128, n0);
                    if (sf) {
                        const uint32_t st = base + L::OFF_SF + stage * 1024;
                        const int64_t g = static_cast<int64_t>(kb >> 2) * 512;
                        q8::bulk_load(st, sw + g, 512u, bar);
                        q8::bulk_load(st + 512u, sx + g, 512u, bar);
                    }
                    ptx::tma_load_2d(at + ROWS * 128, &tm_x, bar, kb * 128, static_cast<int32_t>(t0));
                    issued |= 1u << stage;
                    last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == L::STAGES) stage = 0, phase ^= 1u;
                }
            }
            for (int s = 0; s < L::STAGES; ++s)
                if ((issued >> s) & 1u) wt.wait(full + 8u * s, (last_parity >> s) & 1u, q8::SITE_TEARDOWN, -1, true);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, sf_buf = 0, sfa = 0, n = 0;
            for (int tile = first; tile < p.tiles && ok; tile += step, ++n) {
                const uint32_t acc = n & 1u;
                // the tokens' scales are a tile of 128 rows, 32 to a column: the second
                // 64 tokens of it start two columns in
                const uint32_t sfb_at = 4u + (NT == 64 ? static_cast<uint32_t>(tile / p.tiles_n & 1) * 2u : 0u);
                if (n >= 2 && !wt.wait(acc_free + 8u * acc, ((n >> 1) - 1u) & 1u, q8::SITE_ACC_FREE, tile)) break;
                ptx::tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wt.wait(full + 8u * stage, phase, q8::SITE_FULL, tile)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (kb == kb0 || (kb & 3) == 0) {
                        const uint64_t sd = q8::scale_desc(base + L::OFF_SF + stage * 1024);
                        sfa = tmem + L::SF_COL + sf_buf * 8u;
                        if (++sf_buf == L::SF_BUFS) sf_buf = 0;
                        q8::copy_scales(sfa, sd);
                        q8::copy_scales(sfa + 4u, sd + 32u);
                    }
                    const uint32_t at = base + stage * L::STAGE;
                    const uint64_t a0 = ptx::smem_desc_sw128(at, 16, 1024);
                    const uint64_t b0 = ptx::smem_desc_sw128(at + ROWS * 128, 16, 1024);
                    const uint32_t idesc = p.idesc | q8::scale_id(static_cast<uint32_t>(kb) & 3u);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        q8::mma_mxf8(tmem + acc * L::ACC, a0 + 2u * k, b0 + 2u * k, idesc, sfa, sfa + sfb_at,
                                     (kb > kb0 || k > 0) ? 1u : 0u);
                    ptx::mma_commit(empty + 8u * stage);
                    if (++stage == L::STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                ptx::mma_commit(acc_full + 8u * acc);
            }
            // every MMA has completed before shared and tensor memory go
            ptx::mma_commit(teardown);
            wt.wait(teardown, 0u, q8::SITE_TEARDOWN, -1, true);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        // token t belongs to rank t % splits, as its token t / splits
        const int owned = (NT + p.splits - 1) / p.splits;
        const uint32_t part = base + L::OFF_PART + static_cast<uint32_t>((rank * owned * ROWS + row) * 4);
        const int shift = __ffs(p.splits) - 1;
        uint32_t n = 0;
        for (int tile = first; tile < p.tiles; tile += step, ++n) {
            const int64_t o = static_cast<int64_t>(tile % p.tiles_n) * ROWS + row;
            const int64_t t0 = static_cast<int64_t>(tile / p.tiles_n) * NT;
            const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), p.T - t0));
            const bool in = o < p.N;
            float b = 0.f;
            if (p.bias && in && p.splits == 1)
                b = p.f32 ? static_cast<const float*>(p.bias)[o] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[o]);
            const uint32_t acc = n & 1u;
            if (!wt.wait_warp(acc_full + 8u * acc, (n >> 1) & 1u, q8::SITE_ACC_FULL, tile)) break;
            ptx::tc_fence_after();
            const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * L::ACC;
#pragma unroll 1
            for (int c = 0; c < tokens; c += 16) {
                uint32_t v[16];
                q8::tmem_ld16(src + c, v);
                if (p.splits > 1) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = c + e;
                        if (t < tokens)
                            ptx::st_dsmem_u32(ptx::mapa(part + static_cast<uint32_t>(t >> shift) * (ROWS * 4u),
                                                        static_cast<uint32_t>(t & (p.splits - 1))),
                                              v[e]);
                    }
                } else if (in) {
                    if (p.f32) {
                        float* dst = static_cast<float*>(p.out) + (t0 + c) * p.N + o;
#pragma unroll
                        for (int e = 0; e < 16; ++e, dst += p.N)
                            if (c + e < tokens) *dst = __uint_as_float(v[e]) + b;
                    } else {
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (t0 + c) * p.N + o;
#pragma unroll
                        for (int e = 0; e < 16; ++e, dst += p.N)
                            if (c + e < tokens) *dst = __float2bfloat16_rn(__uint_as_float(v[e]) + b);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(acc_free + 8u * acc);
        }
    }
    if (p.splits > 1) {
        ptx::cluster_sync();  // this rank's tokens have every rank's partial sums
        const int64_t o = static_cast<int64_t>(first % p.tiles_n) * ROWS + 4 * lane;  // (N is a multiple of 4)
        const int64_t t0 = static_cast<int64_t>(first / p.tiles_n) * NT;
        const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), p.T - t0));
        const int owned = (NT + p.splits - 1) / p.splits;
        if (o < p.N) {
            float b[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.bias) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[e] = p.f32 ? static_cast<const float*>(p.bias)[o + e] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[o + e]);
            }
            for (int i = warp; rank + i * p.splits < tokens; i += THREADS / 32) {
                const uint32_t at = base + L::OFF_PART + static_cast<uint32_t>((i * ROWS + 4 * lane) * 4);
                float4 f[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < p.splits) f[s] = ptx::lds128f(at + static_cast<uint32_t>(s * owned * ROWS * 4));
                float4 v = f[0];
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    if (s < p.splits) v.x += f[s].x, v.y += f[s].y, v.z += f[s].z, v.w += f[s].w;
                const int64_t to = (t0 + rank + i * p.splits) * p.N + o;
                v.x += b[0], v.y += b[1], v.z += b[2], v.w += b[3];
                if (p.f32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = v;
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

bool encode(CUtensorMap* m, const void* base, uint64_t ld, uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = get_encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {ld, rows}, strides[1] = {ld};
    const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of 2, 4 and 8 CTAs that can be resident at once on a device; 0: unknown.
struct Device {
    int done = 0, clusters[9] = {};
};

template <int NT>
cudaError_t launch(const Q8Product& q, Params p, int num_sms, cudaStream_t stream) {
    static std::mutex m;
    static Device devices[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg<NT>::SMEM;
    cfg.attrs = attr;
    std::lock_guard<std::mutex> g(m);
    Device& d = devices[dev];
    if (!d.done) {
        e = cudaFuncSetAttribute(q8_tokens_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::SMEM);
        if (e != cudaSuccess) return e;
        for (int s = 2; s <= 8; s *= 2) {
            cfg.gridDim = dim3(static_cast<unsigned>(s), 1, 1);
            cfg.numAttrs = 1;
            attr[0].val.clusterDim.x = static_cast<unsigned>(s);
            if (cudaOccupancyMaxActiveClusters(&d.clusters[s], q8_tokens_kernel<NT>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                d.clusters[s] = 0;
            }
        }
        d.done = 1;
    }
    // as many ranks as leave every cluster resident (a second wave costs more than
    // the shorter K saves) and two blocks of K to each
    int splits = 1;
    while (splits < 8 && 4 * splits <= p.kb && p.tiles <= d.clusters[2 * splits]) splits *= 2;
    if (const char* t = std::getenv("MMBWD_Q8_TOKEN_SPLITS")) {  // tuning and tests
        const int s = std::atoi(t);
        if ((s == 1 || s == 2 || s == 4 || s == 8) && s <= p.kb) splits = s;
    }
    CUtensorMap w, x;
    const uint64_t ld = static_cast<uint64_t>(q8_ld(q.K));
    if (!encode(&w, q.B, ld, static_cast<uint64_t>(q.N), ROWS) || !encode(&x, q.A, ld, static_cast<uint64_t>(q.M), NT))
        return cudaErrorInvalidValue;
    p.splits = splits;
    p.idesc = q8::idesc_mxf8(ROWS, NT, q.b_format, q.a_format);
    cfg.gridDim = dim3(static_cast<unsigned>(splits > 1 ? p.tiles * splits : std::min(p.tiles, 2 * num_sms)), 1, 1);
    cfg.stream = stream;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q8_tokens_kernel<NT>, w, x, p);
}

}  // namespace

cudaError_t q8_tokens_launch(const Q8Product& q, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    Params p{};
    p.out = q.D, p.bias = q.bias, p.w_scale = q.b_scale, p.x_scale = q.a_scale;
    p.T = q.M, p.N = q.N, p.groups = q8_groups(q.K);
    p.kb = static_cast<int>(q8_blocks(q.K));
    p.f32 = q.dtype == MMBWD_F32 ? 1 : 0;
    p.wait_ns = q8_wait_limit_ns();
    p.tiles_n = static_cast<int>((q.N + ROWS - 1) / ROWS);
    const int64_t tiles = p.tiles_n * (q.M <= 64 ? 1 : (q.M + 63) / 64);
    if (tiles > INT32_MAX / 8) return cudaErrorInvalidValue;
    p.tiles = static_cast<int>(tiles);
    if (q.M <= 16) return launch<16>(q, p, num_sms, stream);
    if (q.M <= 32) return launch<32>(q, p, num_sms, stream);
    return launch<64>(q, p, num_sms, stream);
}

__global__ void q8_tokens_selftest_kernel(unsigned long long limit_ns) {
    q8::selftest_wait(g_q8_tokens_status, limit_ns);
}

cudaError_t q8_tokens_selftest_wait(unsigned long long limit_ns) {
    q8_tokens_selftest_kernel<<<1, 1>>>(limit_ns);
    return cudaGetLastError();
}

cudaError_t q8_tokens_read_status(int* code, int* info3, bool reset) {
    unsigned int h[4] = {0, 0, 0, 0};
    cudaError_t e = cudaMemcpyFromSymbol(h, g_q8_tokens_status, sizeof(h));
    if (e != cudaSuccess) return e;
    *code = h[0] ? -static_cast<int>(h[0]) : MMBWD_OK;
    for (int i = 0; i < 3; ++i) info3[i] = static_cast<int>(h[1 + i]);
    if (reset) {
        const unsigned int z[4] = {0, 0, 0, 0};
        e = cudaMemcpyToSymbol(g_q8_tokens_status, z, sizeof(z));
    }
    return e;
}

}  // namespace mmbwd
