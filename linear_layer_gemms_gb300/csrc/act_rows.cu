// Activations by themselves (include/linear_epilogue.h): the gradient through one, element
// by element, and the forward of a layer that has no inputs (C == 0).
#include "act.cuh"
#include "ops.h"
#include "ptx.cuh"

#include <algorithm>

namespace mmbwd {
namespace {

constexpr int THREADS = 256;
constexpr int VECS = 4;  // 16-byte vectors of each tensor in flight to a thread

template <typename T, int ACT>
__device__ __forceinline__ uint4 slope_product(const uint4& d, const uint4& x) {
    const uint32_t a[4] = {d.x, d.y, d.z, d.w}, b[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            float lo = __uint_as_float(a[i] << 16), hi = __uint_as_float(a[i] & 0xFFFF0000u);
            act::slope_fast<ACT>(lo, hi, __uint_as_float(b[i] << 16), __uint_as_float(b[i] & 0xFFFF0000u));
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            r[i] = __float_as_uint(__uint_as_float(a[i]) * act::slope<ACT>(__uint_as_float(b[i])));
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// dpre = dout * act'(pre): bound by HBM, two reads and a write of each value. dpre may be
// dout or pre: a thread has read what it writes. No activation: no pre, a copy of dout.
template <typename T>
__global__ void __launch_bounds__(THREADS) act_backward_kernel(T* dpre, const T* dout, const T* pre, int64_t n, int act) {
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int PER = 16 / sizeof(T);
    const int64_t vecs = n / PER;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (THREADS * VECS) + threadIdx.x;
    const uint4 *d4 = reinterpret_cast<const uint4*>(dout), *x4 = reinterpret_cast<const uint4*>(pre);
    uint4* o4 = reinterpret_cast<uint4*>(dpre);
    uint4 d[VECS], x[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j)
        if (at + j * THREADS < vecs) {
            d[j] = d4[at + j * THREADS];
            x[j] = pre ? x4[at + j * THREADS] : make_uint4(0u, 0u, 0u, 0u);
        }
    act::with(act, [&](auto a) {
#pragma unroll
        for (int j = 0; j < VECS; ++j)
            if (at + j * THREADS < vecs) o4[at + j * THREADS] = slope_product<T, decltype(a)::value>(d[j], x[j]);
        const int64_t i = vecs * PER + at;  // the loose values at the end: the first threads'
        if (i < n) {
            float v = static_cast<float>(dout[i]), unused = 0.f;
            const float x = pre ? static_cast<float>(pre[i]) : 0.f;
            if constexpr (sizeof(T) == 2) act::slope_fast<decltype(a)::value>(v, unused, x, 0.f);
            else v *= act::slope<decltype(a)::value>(x);
            dpre[i] = static_cast<T>(v);
        }
    });
}

// pre = bias, out = act(bias) + residual
template <typename T>
__global__ void __launch_bounds__(THREADS) act_rows_kernel(T* out, T* pre, const T* bias, const T* residual, int64_t n,
                                                           int64_t cols, int act) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * THREADS) {
        const float s = bias ? static_cast<float>(bias[i % cols]) : 0.f;
        act::with(act, [&](auto a) {
            float v = s, unused = 0.f;
            if constexpr (sizeof(T) == 2) act::value_fast<decltype(a)::value>(v, unused);
            else v = act::value<decltype(a)::value>(v);
            if (residual) v += static_cast<float>(residual[i]);
            out[i] = static_cast<T>(v);
        });
        if (pre) pre[i] = static_cast<T>(s);
    }
}

template <typename T>
cudaError_t launch_backward(T* dpre, const T* dout, const T* pre, int64_t n, int act, cudaStream_t stream) {
    const int64_t vecs = std::max<int64_t>(1, n / (16 / static_cast<int64_t>(sizeof(T))));
    const int64_t blocks = (vecs + THREADS * VECS - 1) / (THREADS * VECS);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, act_backward_kernel<T>, dpre, dout, pre, n, act);
}

}  // namespace

cudaError_t act_backward_launch(void* dpre, const void* dout, const void* pre, int64_t n, int act, int dtype,
                                cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    if (dtype == MMBWD_F32)
        return launch_backward(static_cast<float*>(dpre), static_cast<const float*>(dout), static_cast<const float*>(pre),
                               n, act, stream);
    return launch_backward(static_cast<__nv_bfloat16*>(dpre), static_cast<const __nv_bfloat16*>(dout),
                           static_cast<const __nv_bfloat16*>(pre), n, act, stream);
}

cudaError_t act_rows_launch(void* out, void* pre, const void* bias, const void* residual, int64_t rows, int64_t cols,
                            int act, int dtype, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    const int64_t n = rows * cols;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((n + THREADS - 1) / THREADS, 4096));
    if (dtype == MMBWD_F32)
        act_rows_kernel<<<blocks, THREADS, 0, stream>>>(static_cast<float*>(out), static_cast<float*>(pre),
                                                        static_cast<const float*>(bias), static_cast<const float*>(residual),
                                                        n, cols, act);
    else
        act_rows_kernel<<<blocks, THREADS, 0, stream>>>(
            static_cast<__nv_bfloat16*>(out), static_cast<__nv_bfloat16*>(pre), static_cast<const __nv_bfloat16*>(bias),
            static_cast<const __nv_bfloat16*>(residual), n, cols, act);
    return cudaGetLastError();
}

}  // namespace mmbwd
