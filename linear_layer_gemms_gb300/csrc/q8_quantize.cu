// Quantisation into the 8-bit form of include/q8_linear.h: blocks of 128 values
// with a power-of-two scale, along the rows (row form), along the columns
// (column form: the 8-bit form of the transposed matrix), or both from one
// read of x, with the column sums of x on request.
//
// Bound by HBM: es bytes read and one byte written per element and form. A
// block of 256 threads takes a 128 x 128 tile, so that one tile holds whole
// blocks of both directions. Thread (g, u) = (tid / 16, tid % 16) keeps rows
// 8g .. 8g+7 of columns 8u .. 8u+7 in registers: a row's maximum is then four
// shuffles over the 16 lanes that share the row; a column's maximum goes over
// the eight rows in registers, one shuffle, and a shared-memory atomic maximum
// across the eight warps (exact, so its order does not matter). The column
// form's bytes are turned through shared memory (16 KB; the 8-byte granule g
// of column c at g ^ (c / 8), free of bank conflicts in both directions) and
// written as 128 contiguous bytes per column.
#include "../../include/q8_linear.h"
#include "ops.h"
#include "ptx.cuh"
#include "q8.h"

#include <cuda_bf16.h>

namespace mmbwd {
namespace {

constexpr int QT_THREADS = 256;

template <int FMT>
struct Fmt;
template <>
struct Fmt<MMBWD_E4M3> {
    static constexpr int EMAX = 8;  // largest value 1.75 * 2^8
    __device__ static uint32_t pack2(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Fmt<MMBWD_E5M2> {
    static constexpr int EMAX = 15;  // largest value 1.75 * 2^15
    __device__ static uint32_t pack2(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// Scale byte (s + 127) of a block whose largest finite magnitude is amax >= 0:
// both formats' largest value is 1.75 * 2^EMAX, so amax = m * 2^p (m in [1, 2))
// needs s = p - EMAX, one more when m > 1.75.
template <int FMT>
__device__ __forceinline__ int scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b == 0u) return 127;
    const int s = static_cast<int>(b >> 23) - 127 - Fmt<FMT>::EMAX + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return s < -127 ? 0 : s + 127;
}

// 2^-s of a scale byte (s in -127 .. 120, so the result is a normal number).
__device__ __forceinline__ float inv_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }

// Eight consecutive values of a row, as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void load(const __nv_bfloat16* p, int64_t left) {  // left >= 1: whole vectors remain
        a = left >= 8 ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void load(const float* p, int64_t left) {
        a = left >= 4 ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b = left >= 8 ? __ldcs(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

template <typename T, int FMT, bool ROW, bool COL>
__global__ void __launch_bounds__(QT_THREADS) q8_quantize_kernel(uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                                 uint8_t* __restrict__ qt, uint8_t* __restrict__ scale_t,
                                                                 float* __restrict__ partials, const T* __restrict__ x,
                                                                 int64_t rows, int64_t cols, int64_t ld, int64_t ldt,
                                                                 int64_t kb_row, int64_t kb_col, int64_t tiles_c) {
    using F = Fmt<FMT>;
    __shared__ uint32_t col_max[128];
    __shared__ float col_inv[128];
    __shared__ __align__(16) uint8_t turned[COL ? 128 * 128 : 16];
    __shared__ float sums[8][128];
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5;
    const int g = tid >> 4, u = tid & 15;
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;  // the tile: row block, column block
    const int64_t r0 = tr * 128, c0 = tc * 128;
    if (COL && tid < 128) col_max[tid] = 0u;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();

    Raw8<T> raw[8];
    const int64_t c = c0 + 8 * u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * g + i;
        raw[i].zero();
        if (r < rows && c < cols) raw[i].load(x + r * cols + c, cols - c);
    }

    float cmax[8], csum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = csum[j] = 0.f;
    int my_scale = 127;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        raw[i].get(f);
        float m = 0.f;
        if (partials) {
#pragma unroll
            for (int j = 0; j < 8; ++j) csum[j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = finite(f[j]) ? fabsf(f[j]) : 0.f;
            m = fmaxf(m, a);
            if (COL) cmax[j] = fmaxf(cmax[j], a);
        }
        if constexpr (ROW) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int sb = scale_byte<FMT>(m);
            if (u == i) my_scale = sb;
            const float inv = inv_scale(sb);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (inf * 2^-s stays inf: stored as the format's NaN)
                const float a = finite(f[2 * j]) ? f[2 * j] * inv : __uint_as_float(0x7FFFFFFFu);
                const float b = finite(f[2 * j + 1]) ? f[2 * j + 1] * inv : __uint_as_float(0x7FFFFFFFu);
                w[j] = F::pack2(a, b);
            }
            const int64_t r = r0 + 8 * g + i;
            if (r < rows && c < ld)
                *reinterpret_cast<uint2*>(q + r * ld + c) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        }
    }
    if constexpr (ROW) {
        const int64_t groups = (kb_row + 3) / 4;
        const int rl = 8 * g + u;  // lanes u < 8 hold one row's scale each
        uint8_t* at = scale + (tr * groups + tc / 4) * 512 + (rl % 32) * 16 + (rl / 32) * 4;
        if (u < 8) {
            at[tc % 4] = static_cast<uint8_t>(my_scale);
            if (tc == kb_row - 1)
                for (int64_t k = tc % 4 + 1; k < 4; ++k) at[k] = 127;
        }
    }
    if (partials) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = csum[j] + __shfl_down_sync(0xffffffffu, csum[j], 16);
            if ((tid & 31) < 16) sums[warp][8 * u + j] = s;
        }
    }
    if (COL || partials) __syncthreads();
    if (partials && tid < 128 && c0 + tid < cols) {
        float s = sums[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sums[w][tid];
        partials[tr * cols + c0 + tid] = s;
    }
    if constexpr (COL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));
            if ((tid & 31) < 16) atomicMax(&col_max[8 * u + j], __float_as_uint(m));
        }
        __syncthreads();
        if (tid < 128) {
            const int sb = scale_byte<FMT>(__uint_as_float(col_max[tid]));
            col_inv[tid] = inv_scale(sb);
            const int64_t groups = (kb_col + 3) / 4;
            uint8_t* at = scale_t + (tc * groups + tr / 4) * 512 + (tid % 32) * 16 + (tid / 32) * 4;
            at[tr % 4] = static_cast<uint8_t>(sb);
            if (tr == kb_col - 1)
                for (int64_t k = tr % 4 + 1; k < 4; ++k) at[k] = 127;
        }
        __syncthreads();
        uint32_t w[8][2];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float f0[8], f1[8];
            raw[i].get(f0);
            raw[i + 1].get(f1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float inv = col_inv[8 * u + j];
                const float a = finite(f0[j]) ? f0[j] * inv : __uint_as_float(0x7FFFFFFFu);
                const float b = finite(f1[j]) ? f1[j] * inv : __uint_as_float(0x7FFFFFFFu);
                const uint32_t p = F::pack2(a, b);
                w[j][i / 4] = (i % 4) ? w[j][i / 4] | (p << 16) : p;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint2*>(turned + (8 * u + j) * 128 + ((g ^ u) << 3)) = make_uint2(w[j][0], w[j][1]);
        __syncthreads();
        const int h = tid & 7;
        const int64_t rr = r0 + 16 * h;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int cl = 32 * it + (tid >> 3);
            const uint8_t* row = turned + cl * 128;
            const uint2 a = *reinterpret_cast<const uint2*>(row + (((2 * h) ^ (cl >> 3)) << 3));
            const uint2 b = *reinterpret_cast<const uint2*>(row + (((2 * h + 1) ^ (cl >> 3)) << 3));
            if (c0 + cl < cols && rr < ldt)
                *reinterpret_cast<uint4*>(qt + (c0 + cl) * ldt + rr) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
}

// colsum[c] = the row blocks' sums added in order: eight warps of a block each
// take a contiguous eighth of the row blocks for 32 columns, then the eighths
// are added in order and rounded once.
template <typename T>
__global__ void __launch_bounds__(256) q8_colsum_kernel(T* __restrict__ colsum, const float* __restrict__ partials,
                                                        int64_t nblocks, int64_t cols) {
    __shared__ float part[8][32];
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int64_t per = (nblocks + 7) / 8, b0 = warp * per, b1 = b0 + per < nblocks ? b0 + per : nblocks;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t b = b0; b < b1; ++b) s += __ldcg(partials + b * cols + c);
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = part[0][lane];
#pragma unroll
        for (int w = 1; w < 8; ++w) t += part[w][lane];
        if constexpr (sizeof(T) == 4)
            colsum[c] = t;
        else
            colsum[c] = __float2bfloat16_rn(t);
    }
}

template <typename T, int FMT, bool ROW, bool COL>
cudaError_t launch_tiles(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, float* partials, const T* x,
                         int64_t rows, int64_t cols, cudaStream_t stream) {
    const int64_t tiles_r = q8_blocks(rows), tiles_c = q8_blocks(cols);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles_r * tiles_c), 1, 1);
    cfg.blockDim = dim3(QT_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q8_quantize_kernel<T, FMT, ROW, COL>, q, scale, qt, scale_t, partials, x, rows,
                              cols, q8_ld(cols), q8_ld(rows), q8_blocks(cols), q8_blocks(rows), tiles_c);
}

template <typename T, int FMT>
cudaError_t launch_forms(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* colsum, const T* x,
                         float* partials, int64_t rows, int64_t cols, cudaStream_t stream) {
    float* part = colsum ? partials : nullptr;
    cudaError_t e;
    if (q && qt)
        e = launch_tiles<T, FMT, true, true>(q, scale, qt, scale_t, part, x, rows, cols, stream);
    else if (qt)
        e = launch_tiles<T, FMT, false, true>(q, scale, qt, scale_t, part, x, rows, cols, stream);
    else
        e = launch_tiles<T, FMT, true, false>(q, scale, qt, scale_t, part, x, rows, cols, stream);
    if (e != cudaSuccess || !colsum) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((cols + 31) / 32), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q8_colsum_kernel<T>, static_cast<T*>(colsum),
                              static_cast<const float*>(partials), q8_blocks(rows), cols);
}

}  // namespace

cudaError_t q8_quantize_launch(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* colsum, const void* x,
                               float* partials, int64_t rows, int64_t cols, int dtype, int format,
                               cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    if (dtype == MMBWD_F32) {
        const float* p = static_cast<const float*>(x);
        return format == MMBWD_E4M3 ? launch_forms<float, MMBWD_E4M3>(q, scale, qt, scale_t, colsum, p, partials, rows, cols, stream)
                                    : launch_forms<float, MMBWD_E5M2>(q, scale, qt, scale_t, colsum, p, partials, rows, cols, stream);
    }
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x);
    return format == MMBWD_E4M3 ? launch_forms<__nv_bfloat16, MMBWD_E4M3>(q, scale, qt, scale_t, colsum, p, partials, rows, cols, stream)
                                : launch_forms<__nv_bfloat16, MMBWD_E5M2>(q, scale, qt, scale_t, colsum, p, partials, rows, cols, stream);
}

}  // namespace mmbwd
