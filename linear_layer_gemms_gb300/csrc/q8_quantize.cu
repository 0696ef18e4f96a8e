// Quantisation into the 8-bit form of include/q8_linear.h: blocks of 128 values
// with a power-of-two scale, along the rows (row form), along the columns
// (column form: the 8-bit form of the transposed matrix), or both from one
// read of x, with the column sums of x on request.
//
// Bound by HBM: es bytes read and one byte written per element and form (31 us
// for 8192 x 6400 bf16 into both forms at the measured copy rate). A block of 256
// threads takes a 128 x 128 tile, so that one tile holds whole blocks of both
// directions. Thread (g, u) = (tid / 16, tid % 16) keeps rows 8g .. 8g+7 of
// columns 8u .. 8u+7 in registers as they are stored: a row's maximum is then four
// shuffles over the 16 lanes that share the row (two rows to a word in bf16); a
// column's maximum goes over the eight rows in registers, one shuffle, and a
// shared-memory atomic maximum across the eight warps (exact, so its order does
// not matter). The column form's bytes are turned through shared memory (16 KB; the
// 8-byte granule g of column c at g ^ (c / 8), free of bank conflicts in both
// directions) and written as 128 contiguous bytes per column.
//
// Next to the bytes the instruction count is the limit, so the inner steps are
// chosen for few instructions (13 per value, both forms and sums): maxima by
// max.xorsign.abs (no sign masks; a NaN wins, which is how a tile with a
// non-finite value is found and sent down a path of its own), scales by one
// carrying addition, bf16 halves multiplied and summed into fp32 without
// unpacking them, four conversions packed into a word at once. 8192 x 6400 bf16:
// both forms 34.6 us (6.1 TB/s, 0.90 of the copy rate), with the column sums 37.4;
// the first version, with a finiteness test per value, took 104 and 110. Four blocks
// an SM against three: 36.4 against 40 (before the last steps).
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
    // four values, the first in the lowest byte
    __device__ static uint32_t pack4(float a, float b, float c, float d) {
        uint32_t r;
        asm("{.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
            "mov.b32 %0, {x, y};}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    }
};
template <>
struct Fmt<MMBWD_E5M2> {
    static constexpr int EMAX = 15;  // largest value 1.75 * 2^15
    // four values, the first in the lowest byte
    __device__ static uint32_t pack4(float a, float b, float c, float d) {
        uint32_t r;
        asm("{.reg .b16 x, y;\n\tcvt.rn.satfinite.e5m2x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 y, %4, %3;\n\t"
            "mov.b32 %0, {x, y};}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    }
};

// Scale byte (s + 127) of a block whose largest finite magnitude has the fp32
// bits b: both formats' largest value is 1.75 * 2^EMAX, so amax = m * 2^p (m in
// [1, 2)) needs s = p - EMAX, one more when m > 1.75: adding 0x1FFFFF to the
// bits carries into the exponent exactly then.
template <int FMT>
__device__ __forceinline__ int scale_byte(uint32_t b) {
    if (b == 0u) return 127;
    const int e = static_cast<int>((b + 0x1FFFFFu) >> 23) - Fmt<FMT>::EMAX;
    return e < 0 ? 0 : e;
}

// 2^-s of the same block, as fp32 bits (s in -127 .. 120: a normal number). A
// block of zeros gets the largest, which leaves them zeros.
template <int FMT>
__device__ __forceinline__ uint32_t inv_scale(uint32_t b) {
    constexpr uint32_t LOW = static_cast<uint32_t>(Fmt<FMT>::EMAX) << 23, TOP = static_cast<uint32_t>(254 + Fmt<FMT>::EMAX) << 23;
    const uint32_t t = b + 0x1FFFFFu;
    return TOP - ((t > LOW ? t : LOW) & 0xFF800000u);
}
// The same for two bf16 magnitudes in one word, as a bf16 pair.
template <int FMT>
__device__ __forceinline__ uint32_t inv_scale2(uint32_t p) {
    constexpr uint32_t LOW = (Fmt<FMT>::EMAX << 7) * 0x00010001u, TOP = ((254 + Fmt<FMT>::EMAX) << 7) * 0x00010001u;
    return TOP - (__vmaxu2(p + 0x001F001Fu, LOW) & 0xFF80FF80u);
}

__device__ __forceinline__ uint32_t lo_bf16(uint32_t w) { return w << 16; }
__device__ __forceinline__ uint32_t hi_bf16(uint32_t w) { return w & 0xFFFF0000u; }

// Eight consecutive values of a row as they are stored: W words. larger():
// per value the larger magnitude of two, a NaN if either is one; its sign
// means nothing (max.NaN.xorsign.abs takes magnitudes without extra instructions).
template <typename T>
struct Eight;

template <>
struct Eight<__nv_bfloat16> {
    static constexpr int W = 4;  // two values a word
    static constexpr uint32_t MAG = 0x7FFF7FFFu;
    uint32_t w[4];
    __device__ void load(const __nv_bfloat16* p, int left) {  // left: values up to the row's end, <= 0: none
        const uint4 a = left >= 8 ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    }
    __device__ static uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // whether a maximum (sign cleared) is an infinity or a NaN
    __device__ static bool bad(uint32_t m) { return (m & 0xFFFFu) >= 0x7F80u || (m >> 16) >= 0x7F80u; }
    // value e of eight maxima, as fp32 bits
    __device__ static uint32_t bits(const uint32_t (&m)[4], int e) { return e & 1 ? hi_bf16(m[e >> 1]) : lo_bf16(m[e >> 1]); }
    __device__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(lo_bf16(w[i])), f[2 * i + 1] = __uint_as_float(hi_bf16(w[i]));
    }
};

template <>
struct Eight<float> {
    static constexpr int W = 8;
    static constexpr uint32_t MAG = 0x7FFFFFFFu;
    uint32_t w[8];
    __device__ void load(const float* p, int left) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        const uint4 a = left >= 4 ? __ldcs(reinterpret_cast<const uint4*>(p)) : z;
        const uint4 b = left >= 8 ? __ldcs(reinterpret_cast<const uint4*>(p) + 1) : z;
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    __device__ static uint32_t larger(uint32_t a, uint32_t b) {
        float r;
        asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(r);
    }
    __device__ static bool bad(uint32_t m) { return m >= 0x7F800000u; }
    __device__ static uint32_t bits(const uint32_t (&m)[8], int e) { return m[e]; }
    __device__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
};

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// A tile's shared memory.
struct TileMem {
    uint32_t col_max[128];
    uint32_t col_inv[128];  // 2^-s as fp32 bits
    float sums[8][128];
    alignas(16) uint8_t turned[128 * 128];
};

// Products and sums of a bf16 half of a word in fp32, one instruction each
// without unpacking it (x * s - 0: exact, and keeps the sign of a zero).
template <int HALF>
__device__ __forceinline__ float mul_half(uint32_t w, uint32_t s) {
    float r;
    if constexpr (HALF == 0)
        asm("{.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 {c, d}, %2;\n\tfma.rn.f32.bf16 %0, a, c, %3;}"
            : "=f"(r) : "r"(w), "r"(s), "f"(-0.0f));
    else
        asm("{.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 {c, d}, %2;\n\tfma.rn.f32.bf16 %0, b, d, %3;}"
            : "=f"(r) : "r"(w), "r"(s), "f"(-0.0f));
    return r;
}
template <int HALF>
__device__ __forceinline__ float add_half(uint32_t w, float acc) {
    float r;
    if constexpr (HALF == 0)
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, a, %2;}" : "=f"(r) : "r"(w), "f"(acc));
    else
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, b, %2;}" : "=f"(r) : "r"(w), "f"(acc));
    return r;
}

// Values 2i, 2i+1 of `v` times two scales given as fp32 bits (bf16: as a bf16
// pair in s0): exact, the scales being powers of two. RARE: a product that is
// not finite becomes a NaN.
template <typename T, bool RARE>
__device__ __forceinline__ void two(const Eight<T>& v, int i, uint32_t s0, uint32_t s1, float& a, float& b) {
    if constexpr (sizeof(T) == 2) {
        a = mul_half<0>(v.w[i], s0), b = mul_half<1>(v.w[i], s0);
    } else {
        a = __uint_as_float(v.w[2 * i]) * __uint_as_float(s0), b = __uint_as_float(v.w[2 * i + 1]) * __uint_as_float(s1);
    }
    if constexpr (RARE) {
        const float n = __uint_as_float(0x7FFFFFFFu);
        a = finite(a) ? a : n, b = finite(b) ? b : n;
    }
}

// The row form of a tile, from registers.
template <typename T, int FMT, bool RARE>
__device__ __forceinline__ void row_form(const Eight<T> (&v)[8], uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                         int64_t tr, int64_t tc, int64_t rows, int64_t ld, int64_t kb) {
    using E = Eight<T>;
    const int tid = static_cast<int>(threadIdx.x), g = tid >> 4, u = tid & 15;
    const int64_t c = tc * 128 + 8 * u, r0 = tr * 128 + 8 * g;
    uint32_t mine = 0;  // maximum of row 8g + u, as fp32 bits
    uint8_t* dst = q + r0 * ld + c;
    // of this thread's eight rows, how many to store
    const int rows_here = c < ld ? static_cast<int>(r0 + 8 <= rows ? 8 : rows - r0) : 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t t[2];  // the two rows' maxima over this thread's values
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const E& x = v[i + e];
            if constexpr (RARE) {
                float f[8], best = 0.f;
                x.get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) best = finite(f[j]) ? fmaxf(best, fabsf(f[j])) : best;
                t[e] = __float_as_uint(best);
                if constexpr (sizeof(T) == 2) t[e] |= t[e] >> 16;
            } else {
                t[e] = E::larger(x.w[0], x.w[1]);
#pragma unroll
                for (int k = 2; k < E::W; ++k) t[e] = E::larger(t[e], x.w[k]);
            }
        }
        uint32_t s0[2];
        if constexpr (sizeof(T) == 2) {  // both rows' maxima in one word through the shuffles
            uint32_t p = E::larger(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[0], t[1], 0x7632));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) p = E::larger(p, __shfl_xor_sync(0xffffffffu, p, o));
            p &= E::MAG;
            if (u == i) mine = lo_bf16(p);
            if (u == i + 1) mine = hi_bf16(p);
            const uint32_t inv = inv_scale2<FMT>(p);
            s0[0] = __byte_perm(inv, 0u, 0x1010), s0[1] = __byte_perm(inv, 0u, 0x3232);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) t[e] = E::larger(t[e], __shfl_xor_sync(0xffffffffu, t[e], o));
                t[e] &= E::MAG;
                if (u == i + e) mine = t[e];
                s0[e] = inv_scale<FMT>(t[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) two<T, RARE>(v[i + e], j, s0[e], s0[e], f[2 * j], f[2 * j + 1]);
            if (i + e < rows_here)
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(Fmt<FMT>::pack4(f[0], f[1], f[2], f[3]), Fmt<FMT>::pack4(f[4], f[5], f[6], f[7]));
            dst += ld;
        }
    }
    if (u < 8) {  // lane u of the sixteen holds row 8g + u
        const int rl = 8 * g + u;
        uint8_t* at = scale + (tr * ((kb + 3) / 4) + tc / 4) * 512 + (rl % 32) * 16 + (rl / 32) * 4;
        at[tc % 4] = static_cast<uint8_t>(scale_byte<FMT>(mine));
        if (tc == kb - 1)
            for (int64_t k = tc % 4 + 1; k < 4; ++k) at[k] = 127;
    }
}

// The column form's bytes of a tile into `turned`, from registers.
template <typename T, int FMT, bool RARE>
__device__ __forceinline__ void turn_columns(const Eight<T> (&v)[8], TileMem& sm) {
    const int tid = static_cast<int>(threadIdx.x), g = tid >> 4, u = tid & 15;
    uint32_t inv[8];  // as fp32 bits; bf16: words 0 .. 3 hold pairs
    *reinterpret_cast<uint4*>(inv) = *reinterpret_cast<const uint4*>(&sm.col_inv[8 * u]);
    *reinterpret_cast<uint4*>(inv + 4) = *reinterpret_cast<const uint4*>(&sm.col_inv[8 * u + 4]);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) inv[j] = __byte_perm(inv[2 * j], inv[2 * j + 1], 0x7632);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // columns 2j and 2j + 1, byte i of each is row i
        const uint32_t i0 = sizeof(T) == 2 ? inv[j] : inv[2 * j], i1 = sizeof(T) == 2 ? 0u : inv[2 * j + 1];
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) two<T, RARE>(v[i], j, i0, i1, lo[i], hi[i]);
        uint8_t* at = sm.turned + (8 * u + 2 * j) * 128 + ((g ^ u) << 3);
        *reinterpret_cast<uint2*>(at) = make_uint2(Fmt<FMT>::pack4(lo[0], lo[1], lo[2], lo[3]), Fmt<FMT>::pack4(lo[4], lo[5], lo[6], lo[7]));
        *reinterpret_cast<uint2*>(at + 128) = make_uint2(Fmt<FMT>::pack4(hi[0], hi[1], hi[2], hi[3]), Fmt<FMT>::pack4(hi[4], hi[5], hi[6], hi[7]));
    }
}

template <typename T, int FMT, bool ROW, bool COL>
__global__ void __launch_bounds__(QT_THREADS, sizeof(T) == 2 ? 4 : 2)
    q8_quantize_kernel(uint8_t* __restrict__ q, uint8_t* __restrict__ scale, uint8_t* __restrict__ qt,
                       uint8_t* __restrict__ scale_t, float* __restrict__ partials, T* __restrict__ colsum,
                       const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld, int64_t ldt, int64_t kb_row,
                       int64_t kb_col, uint32_t tiles_c) {
    using E = Eight<T>;
    __shared__ TileMem sm;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int g = tid >> 4, u = tid & 15;
    // the tile: row block, column block (colsum: the row blocks of a column are a cluster)
    const uint32_t kbc = static_cast<uint32_t>(kb_col);
    const int64_t tr = colsum ? blockIdx.x % kbc : blockIdx.x / tiles_c, tc = colsum ? blockIdx.x / kbc : blockIdx.x % tiles_c;
    const bool sums = partials || colsum;
    const int64_t r0 = tr * 128, c0 = tc * 128;
    if (COL && tid < 128) sm.col_max[tid] = 0u;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();

    E v[8];
    {
        const int64_t c = c0 + 8 * u, r = r0 + 8 * g;
        const T* src = x + r * cols + c;
        const int left = static_cast<int>(c + 8 <= cols ? 8 : cols - c < 0 ? 0 : cols - c);
        if (r + 8 <= rows && left == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i, src += cols) v[i].load(src, 8);
        } else {
            const int rows_here = static_cast<int>(r + 8 <= rows ? 8 : rows - r);
#pragma unroll
            for (int i = 0; i < 8; ++i, src += cols) v[i].load(src, i < rows_here ? left : 0);
        }
    }
    // column maxima of the thread's eight rows; one non-finite value in the tile
    // sends the whole block down the path that looks at every value
    uint32_t cm[E::W];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < E::W; ++k) {
        uint32_t m = E::larger(v[0].w[k], v[1].w[k]);
#pragma unroll
        for (int i = 2; i < 8; ++i) m = E::larger(m, v[i].w[k]);
        cm[k] = m & E::MAG;
        bad |= E::bad(cm[k]);
    }
    if (sums) {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[2 * k] = add_half<0>(v[i].w[k], s[2 * k]);
                    s[2 * k + 1] = add_half<1>(v[i].w[k], s[2 * k + 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] += __uint_as_float(v[i].w[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += __shfl_down_sync(0xffffffffu, s[j], 16);
        if (lane < 16) {
            *reinterpret_cast<float4*>(&sm.sums[warp][8 * u]) = make_float4(s[0], s[1], s[2], s[3]);
            *reinterpret_cast<float4*>(&sm.sums[warp][8 * u + 4]) = make_float4(s[4], s[5], s[6], s[7]);
        }
    }
    if (COL) __syncthreads();  // col_max is zero
    if (COL) {
#pragma unroll
        for (int k = 0; k < E::W; ++k) cm[k] = E::larger(cm[k], __shfl_xor_sync(0xffffffffu, cm[k], 16)) & E::MAG;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // each half warp takes four of the eight columns
            const uint32_t lo = E::bits(cm, e), hi = E::bits(cm, e + 4);
            atomicMax(&sm.col_max[8 * u + e + (lane < 16 ? 0 : 4)], lane < 16 ? lo : hi);
        }
    }
    const bool rare = __syncthreads_or(bad);
    if (COL && rare) {  // the maxima again, over finite values
        if (tid < 128) sm.col_max[tid] = 0u;
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float f[8];
            E t;
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (n == i) t = v[n];
            t.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (finite(f[j])) atomicMax(&sm.col_max[8 * u + j], __float_as_uint(fabsf(f[j])));
        }
        __syncthreads();
    }
    if (sums && tid < 128) {
        float s = sm.sums[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sm.sums[w][tid];
        if (colsum) sm.sums[0][tid] = s;
        else if (c0 + tid < cols) partials[tr * cols + c0 + tid] = s;
    }
    if (COL && tid < 128) {
        const uint32_t m = sm.col_max[tid];
        sm.col_inv[tid] = inv_scale<FMT>(m);
        uint8_t* at = scale_t + (tc * ((kb_col + 3) / 4) + tr / 4) * 512 + (tid % 32) * 16 + (tid / 32) * 4;
        at[tr % 4] = static_cast<uint8_t>(scale_byte<FMT>(m));
        if (tr == kb_col - 1)
            for (int64_t k = tr % 4 + 1; k < 4; ++k) at[k] = 127;
    }
    if constexpr (ROW) {
        if (rare) row_form<T, FMT, true>(v, q, scale, tr, tc, rows, ld, kb_row);
        else row_form<T, FMT, false>(v, q, scale, tr, tc, rows, ld, kb_row);
    }
    if constexpr (COL) {
        __syncthreads();
        if (rare) turn_columns<T, FMT, true>(v, sm);
        else turn_columns<T, FMT, false>(v, sm);
        __syncthreads();
        const int h = tid & 7;
        const int64_t rr = r0 + 16 * h;
        uint8_t* dst = qt + (c0 + (tid >> 3)) * ldt + rr;
        const int cols_here = rr < ldt ? static_cast<int>(c0 + 128 <= cols ? 128 : cols - c0) : 0;
        const int64_t step = 32 * ldt;
#pragma unroll
        for (int it = 0; it < 4; ++it, dst += step) {
            const int cl = 32 * it + (tid >> 3);
            const uint8_t* row = sm.turned + cl * 128;
            const uint2 a = *reinterpret_cast<const uint2*>(row + (((2 * h) ^ (cl >> 3)) << 3));
            const uint2 b = *reinterpret_cast<const uint2*>(row + (((2 * h + 1) ^ (cl >> 3)) << 3));
            if (cl < cols_here) *reinterpret_cast<uint4*>(dst) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    if (colsum) {  // the row blocks' sums, in order, by the first CTA of the cluster
        ptx::cluster_sync();
        if (tr == 0 && tid < 128 && c0 + tid < cols) {
            const uint32_t at = ptx::smem_u32(&sm.sums[0][tid]);
            float t = sm.sums[0][tid];
            for (uint32_t k = 1; k < kbc; ++k) t += __uint_as_float(ptx::ld_dsmem_u32(ptx::mapa(at, k)));
            if constexpr (sizeof(T) == 4)
                colsum[c0 + tid] = t;
            else
                colsum[c0 + tid] = __float2bfloat16_rn(t);
        }
        ptx::cluster_sync();
    }
}

// More than Q8_SUM_CLUSTER row blocks: colsum[c] = their sums added in order, eight warps of a block each
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
cudaError_t launch_tiles(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, float* partials, T* colsum, const T* x,
                         int64_t rows, int64_t cols, cudaStream_t stream) {
    const int64_t tiles_r = q8_blocks(rows), tiles_c = q8_blocks(cols);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles_r * tiles_c), 1, 1);
    cfg.blockDim = dim3(QT_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(colsum ? tiles_r : 1);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = colsum ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q8_quantize_kernel<T, FMT, ROW, COL>, q, scale, qt, scale_t, partials, colsum, x, rows,
                              cols, q8_ld(cols), q8_ld(rows), q8_blocks(cols), q8_blocks(rows),
                              static_cast<uint32_t>(tiles_c));
}

template <typename T, int FMT>
cudaError_t launch_forms(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* colsum, const T* x,
                         float* partials, int64_t rows, int64_t cols, cudaStream_t stream) {
    // few row blocks: their sums meet in a cluster; more: in the workspace
    T* direct = q8_blocks(rows) <= Q8_SUM_CLUSTER ? static_cast<T*>(colsum) : nullptr;
    float* part = colsum && !direct ? partials : nullptr;
    cudaError_t e;
    if (q && qt)
        e = launch_tiles<T, FMT, true, true>(q, scale, qt, scale_t, part, direct, x, rows, cols, stream);
    else if (qt)
        e = launch_tiles<T, FMT, false, true>(q, scale, qt, scale_t, part, direct, x, rows, cols, stream);
    else
        e = launch_tiles<T, FMT, true, false>(q, scale, qt, scale_t, part, direct, x, rows, cols, stream);
    if (e != cudaSuccess || !part) return e;
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
