// Products of matrices in 8-bit form: D (M x N) = A (M x K) . B (N x K)^T with a
// power-of-two scale per block of 128 along K (include/q8_linear.h).
//
// One block of 256 threads forms a 64 x 64 tile of D: 32 values of K at a time
// are decoded to fp32 with their scale into shared memory, and each thread
// accumulates 4 x 4 elements.
#include "../../include/q8_linear.h"
#include "ops.h"
#include "ptx.cuh"
#include "q8.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace mmbwd {
namespace {

constexpr int SP_TILE = 64, SP_K = 32;

__device__ __forceinline__ float q8_value(uint8_t b, int format) {
    uint32_t h;
    const uint16_t two = b;
    if (format == MMBWD_E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(two));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

__device__ __forceinline__ float scale_value(uint8_t b) {
    return b == 0 ? __uint_as_float(1u << 22) : __uint_as_float(static_cast<uint32_t>(b) << 23);
}

struct Operand {
    const uint8_t *q, *scale;
    int64_t rows, ld, groups;
    int format;
};

__device__ __forceinline__ float load_value(const Operand& o, int64_t r, int64_t k, int64_t K) {
    if (r >= o.rows || k >= K) return 0.f;
    const int64_t kb = k / Q8_BLOCK;
    const uint8_t s = o.scale[(r / 128 * o.groups + kb / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + kb % 4];
    return q8_value(o.q[r * o.ld + k], o.format) * scale_value(s);
}

template <typename T>
__global__ void __launch_bounds__(256) q8_product_kernel(T* D, const T* bias, Operand A, Operand B, int64_t K, int add) {
    __shared__ float sa[SP_K][SP_TILE + 1], sb[SP_K][SP_TILE + 1];
    const int tid = static_cast<int>(threadIdx.x);
    const int64_t tiles_n = (B.rows + SP_TILE - 1) / SP_TILE;
    const int64_t m0 = blockIdx.x / tiles_n * SP_TILE, n0 = blockIdx.x % tiles_n * SP_TILE;
    const int ty = tid / 16, tx = tid % 16;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += SP_K) {
        for (int i = tid; i < SP_TILE * SP_K; i += 256) {
            const int r = i / SP_K, k = i % SP_K;
            sa[k][r] = load_value(A, m0 + r, k0 + k, K);
            sb[k][r] = load_value(B, n0 + r, k0 + k, K);
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < SP_K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= A.rows || n >= B.rows) continue;
            float v = acc[i][j];
            if (bias) v += static_cast<float>(bias[n]);
            if (add) v += static_cast<float>(D[m * B.rows + n]);
            D[m * B.rows + n] = static_cast<T>(v);
        }
}

}  // namespace

cudaError_t q8_product_launch(const Q8Product* products, int n, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    for (int i = 0; i < n; ++i) {
        const Q8Product& p = products[i];
        const Operand A{p.A, p.a_scale, p.M, q8_ld(p.K), q8_groups(p.K), p.a_format};
        const Operand B{p.B, p.b_scale, p.N, q8_ld(p.K), q8_groups(p.K), p.b_format};
        const int64_t tiles = ((p.M + SP_TILE - 1) / SP_TILE) * ((p.N + SP_TILE - 1) / SP_TILE);
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e =
            p.dtype == MMBWD_F32
                ? cudaLaunchKernelEx(&cfg, q8_product_kernel<float>, static_cast<float*>(p.D),
                                     static_cast<const float*>(p.bias), A, B, p.K, p.add)
                : cudaLaunchKernelEx(&cfg, q8_product_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16*>(p.D),
                                     static_cast<const __nv_bfloat16*>(p.bias), A, B, p.K, p.add);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mmbwd
