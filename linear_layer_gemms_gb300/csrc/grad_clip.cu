// The global gradient norm over many tensors and clipping (include/grad_clip.h).
//
// Bound by HBM: the norm reads every value once, clipping reads and writes it once
// more. The list travels in the kernel parameters (up to 1024 tensors a launch), cut
// into chunks of 32 KB that the blocks take in turn, the scaling from the list's end, so
// that it begins with what the norm left in L2. A thread sums the squares
// of its (at most 64) values of a chunk in fp32, four sums side by side, and adds that
// to its 64-bit sum; one 64-bit partial per block, joined in block order by whoever
// needs the norm, so no float atomics and the same bits on every call.
//
// A chunk is eight 16-byte loads of a thread, all in flight before the first is used:
// four resident blocks with 64 registers a thread read faster than eight with 32 (205 M
// fp32 values whose norm is below the limit, in place, 140 -> 134 us, 6.1 TB/s). The
// scaling runs with 8 blocks an SM; 4, 16 and 32 cost up to 5%. The same list clipped
// out of place: 375 us for two reads and a write of 0.82 GB (6.6 TB/s), in bf16 192.
#include "../../include/grad_clip.h"
#include "ops.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

namespace mmbwd {
namespace {

constexpr int THREADS = 256;
constexpr int VECS = 8;                                  // 16-byte vectors of a chunk to a thread
constexpr int CHUNK_BYTES = THREADS * VECS * 16;
// The last 80 MB that the norm reads should stay in L2 for the scaling, all else is read and
// written past it (evicted first): 205 M bf16 values 198 -> 192 us, fp32 379 -> 375.
constexpr int KEEP_CHUNKS = (80 << 20) / CHUNK_BYTES;

// The tensors of a launch: tensor t has the chunks first[t] .. first[t + 1).
template <int N>
struct Table {
    void* grad[N];
    void* out[N];
    int64_t count[N];  // values, times 2, plus 1 for bf16
    int first[N + 1];
    int n;
};

struct Values {  // what a chunk covers: `vecs` vectors from `base`, and loose values before and after them
    int64_t base, vecs, head, tail;
};

// Chunk k of a tensor: its vectors start at the tensor's first 16-byte boundary, after
// `head` loose values (chunk 0's); the last chunk has the loose tail.
__device__ __forceinline__ Values chunk_values(uintptr_t p, int64_t count, int es, int64_t k) {
    const int per = 16 / es;
    const int64_t head = min(static_cast<int64_t>((16 - (p & 15)) & 15) / es, count);
    const int64_t all = (count - head) / per;
    Values v;
    v.base = head + k * (CHUNK_BYTES / es);
    v.vecs = min(static_cast<int64_t>(THREADS * VECS), all - k * (THREADS * VECS));
    v.head = k == 0 ? head : 0;
    v.tail = k * (THREADS * VECS) + v.vecs == all ? count - head - all * per : 0;
    return v;
}

template <typename T>
__device__ __forceinline__ float value(const T* p) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
    else return *p;
}

// The squares of a vector's values times `by`^2, onto four sums.
template <typename T>
__device__ __forceinline__ void squares(const uint4& v, float (&s)[4], float by = 1.f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            const float a = __uint_as_float(w[i] << 16) * by, b = __uint_as_float(w[i] & 0xFFFF0000u) * by;
            s[i] = fmaf(a, a, fmaf(b, b, s[i]));
        } else {
            const float a = __uint_as_float(w[i]) * by;
            s[i] = fmaf(a, a, s[i]);
        }
    }
}

// A thread's vectors of a chunk to `f`, all in flight together. `once`: they need not stay
// in L2.
template <typename T, typename F>
__device__ __forceinline__ void for_chunk(const T* p, const Values& c, bool once, F f) {
    const int t = static_cast<int>(threadIdx.x), vecs = static_cast<int>(c.vecs);
    const uint4* src = reinterpret_cast<const uint4*>(p + c.base) + t;
    uint4 v[VECS];
    auto load = [&](auto get) {
#pragma unroll
        for (int j = 0; j < VECS; ++j) v[j] = t + j * THREADS < vecs ? get(src + j * THREADS) : make_uint4(0u, 0u, 0u, 0u);
    };
    if (once) load([](const uint4* q) { return __ldcs(q); });
    else load([](const uint4* q) { return *q; });
#pragma unroll
    for (int j = 0; j < VECS; ++j) f(v[j], j, t + j * THREADS < vecs);
}

// The thread's loose value: thread t the t-th before the vectors, 8 + t the t-th after.
__device__ __forceinline__ int64_t loose_at(const Values& c, int per) {
    const int t = static_cast<int>(threadIdx.x);
    if (t < c.head) return t;
    return t >= 8 && t < 8 + c.tail ? c.base + c.vecs * per + (t - 8) : -1;
}

// A thread's part of a chunk, in 64 bits. Where the fp32 sum is so large that a square
// may have overflowed (an infinity or a NaN among them), or so small that squares may
// have been lost, it is formed again from values scaled by a power of two; that only
// happens to values beyond 2^60 or all below 2^-40.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int64_t count, int64_t k, bool once) {
    constexpr int PER = 16 / sizeof(T);
    const Values c = chunk_values(reinterpret_cast<uintptr_t>(p), count, sizeof(T), k);
    const int64_t at = loose_at(c, PER);
    const float loose = at >= 0 ? value(p + at) : 0.f;
    float s[4] = {loose * loose, 0.f, 0.f, 0.f};
    uint32_t any = 0;
    for_chunk(p, c, once, [&](const uint4& v, int, bool) {
        squares<T>(v, s);
        any |= v.x | v.y;
        any |= v.z | v.w;
    });
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    const uint32_t magnitude = (any & (sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) | (__float_as_uint(loose) & 0x7FFFFFFFu);
    if (sum < 0x1p120f && (sum > 0x1p-80f || magnitude == 0)) return static_cast<double>(sum);
    const float by = sum > 1.f || sum != sum ? 0x1p-80f : 0x1p100f;
    s[0] = (loose * by) * (loose * by);
    s[1] = s[2] = s[3] = 0.f;
    const uint4* src = reinterpret_cast<const uint4*>(p + c.base);
#pragma unroll 1
    for (int64_t j = threadIdx.x; j < c.vecs; j += THREADS) squares<T>(src[j], s, by);
    const double back = by < 1.f ? 0x1p160 : 0x1p-200;
    return static_cast<double>((s[0] + s[1]) + (s[2] + s[3])) * back;
}

// The tensor of chunk `c`.
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& tab, int c) {
    int lo = 0, hi = tab.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The sum of `x` over the block, in a fixed order, in every thread.
__device__ double block_sum(double x) {
    __shared__ double part[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) s += part[w];
    return s;
}

template <int N>
__global__ void __launch_bounds__(THREADS, GRAD_BLOCKS_PER_SM) grad_squares_kernel(const __grid_constant__ Table<N> tab, double* partials) {
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int chunks = tab.first[tab.n], step = static_cast<int>(gridDim.x);
    double s = 0.0;
    int t = static_cast<int>(blockIdx.x) < chunks ? tensor_of(tab, static_cast<int>(blockIdx.x)) : 0;
    for (int c = static_cast<int>(blockIdx.x); c < chunks; c += step) {
        while (c >= tab.first[t + 1]) ++t;
        const int64_t k = c - tab.first[t], count = tab.count[t] >> 1;
        const bool once = c + KEEP_CHUNKS < chunks;
        s += tab.count[t] & 1 ? chunk_squares(static_cast<const __nv_bfloat16*>(tab.grad[t]), count, k, once)
                              : chunk_squares(static_cast<const float*>(tab.grad[t]), count, k, once);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// The norm from the partial sums, the same in every block.
__device__ float norm_of(const double* partials, int n) {
    double s = 0.0;
    for (int i = static_cast<int>(threadIdx.x); i < n; i += THREADS) s += __ldcg(partials + i);
    return static_cast<float>(sqrt(block_sum(s)));
}

__global__ void __launch_bounds__(THREADS) grad_norm_kernel(float* norm, const double* partials, int n) {
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float v = norm_of(partials, n);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(T* out, const T* p, int64_t count, int64_t k, float coef) {
    constexpr int PER = 16 / sizeof(T);
    const Values c = chunk_values(reinterpret_cast<uintptr_t>(p), count, sizeof(T), k);
    auto put = [&](int64_t i) {
        if constexpr (sizeof(T) == 2) out[i] = __float2bfloat16_rn(value(p + i) * coef);
        else out[i] = p[i] * coef;
    };
    const int64_t at = loose_at(c, PER);
    if (at >= 0) put(at);
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) {  // no vector lies on both sides
        for (int64_t i = threadIdx.x; i < c.vecs * PER; i += THREADS) put(c.base + i);
        return;
    }
    uint4* dst = reinterpret_cast<uint4*>(out + c.base) + threadIdx.x;
    for_chunk(p, c, true, [&](const uint4& v, int j, bool there) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) * coef,
                                                               __uint_as_float(w[i] & 0xFFFF0000u) * coef);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                w[i] = __float_as_uint(__uint_as_float(w[i]) * coef);
            }
        }
        if (there) __stcs(dst + j * THREADS, make_uint4(w[0], w[1], w[2], w[3]));
    });
}

// out = coef * g. The norm comes from `n` partial sums (n > 0, or no `given`), and is
// stored to `norm` by block 0 where that is not null, or is `given`.
template <int N>
__global__ void __launch_bounds__(THREADS) grad_scale_kernel(const __grid_constant__ Table<N> tab, const float* given,
                                                             const double* partials, int n, float* norm,
                                                             float max_norm) {
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float total = given ? __ldcg(given) : norm_of(partials, n);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float ratio = max_norm / (total + 1e-6f), coef = ratio >= 1.f ? 1.f : ratio;  // (a NaN stays one)
    const int last = tab.first[tab.n] - 1 - static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
    int t = last >= 0 ? tensor_of(tab, last) : 0;
    for (int c = last; c >= 0; c -= step) {  // backwards: what the norm read last is still in L2
        while (c < tab.first[t]) --t;
        void* out = tab.out[t];
        if (coef == 1.f && out == tab.grad[t]) continue;
        const int64_t k = c - tab.first[t], count = tab.count[t] >> 1;
        if (tab.count[t] & 1)
            scale_chunk(static_cast<__nv_bfloat16*>(out), static_cast<const __nv_bfloat16*>(tab.grad[t]), count, k, coef);
        else
            scale_chunk(static_cast<float*>(out), static_cast<const float*>(tab.grad[t]), count, k, coef);
    }
}

int64_t chunks_of(const GradTensor& t) {
    const int es = t.bf16 ? 2 : 4;
    const int64_t head = std::min<int64_t>(((16 - (reinterpret_cast<uintptr_t>(t.grad) & 15)) & 15) / es, t.count);
    const int64_t vecs = (t.count - head) / (16 / es);
    return std::max<int64_t>(1, (vecs + THREADS * VECS - 1) / (THREADS * VECS));
}

template <int N>
bool fill(Table<N>* tab, const GradTensor* t, int n) {
    int64_t at = 0;
    for (int i = 0; i < n; ++i) {
        tab->grad[i] = const_cast<void*>(t[i].grad);
        tab->out[i] = t[i].out;
        tab->count[i] = t[i].count * 2 + (t[i].bf16 ? 1 : 0);
        tab->first[i] = static_cast<int>(at);
        at += chunks_of(t[i]);
        if (at > INT32_MAX / 2) return false;  // (a chunk's number plus a grid stays an int)
    }
    tab->first[n] = static_cast<int>(at);
    tab->n = n;
    return true;
}

cudaLaunchConfig_t config(int blocks, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// One launch over at most N tensors: the squares (with `partials` to write) or the scaling.
template <int N>
cudaError_t launch(const GradTensor* t, int n, bool scale, const float* given, double* partials, int n_partials,
                   float* norm, float max_norm, int num_sms, int* blocks_out, cudaStream_t stream) {
    static thread_local Table<N> tab;
    if (!fill(&tab, t, n)) return cudaErrorInvalidValue;
    const int most = scale ? num_sms * GRAD_SCALE_BLOCKS_PER_SM : std::min(num_sms * GRAD_BLOCKS_PER_SM, GRAD_MAX_BLOCKS);
    const int blocks = std::max(1, std::min(tab.first[n], most));
    if (blocks_out) *blocks_out = blocks;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(blocks, stream, attr);
    if (!scale) return cudaLaunchKernelEx(&cfg, grad_squares_kernel<N>, tab, partials);
    return cudaLaunchKernelEx(&cfg, grad_scale_kernel<N>, tab, given, static_cast<const double*>(partials), n_partials, norm,
                              max_norm);
}

template <typename... A>
cudaError_t launch_any(const GradTensor* t, int n, A... a) {
    return n <= 32 ? launch<32>(t, n, a...) : n <= 256 ? launch<256>(t, n, a...) : launch<GRAD_TABLE>(t, n, a...);
}

}  // namespace

cudaError_t grad_launch(const GradTensor* list, int n, float* norm, const float* given, bool scale, float max_norm,
                        double* ws, int num_sms, cudaStream_t stream) {
    if (take_injected_launch_failure()) return cudaErrorLaunchFailure;
    int partials = 0;
    if (!given) {
        for (int i = 0; i < n; i += GRAD_TABLE) {
            int blocks = 0;
            const cudaError_t e = launch_any(list + i, std::min(n - i, GRAD_TABLE), false, static_cast<const float*>(nullptr),
                                             ws + partials, 0, static_cast<float*>(nullptr), 0.f, num_sms, &blocks, stream);
            if (e != cudaSuccess) return e;
            partials += blocks;
        }
        if (!scale || n == 0) {
            cudaLaunchAttribute attr[1];
            const cudaLaunchConfig_t cfg = config(1, stream, attr);
            return cudaLaunchKernelEx(&cfg, grad_norm_kernel, norm, static_cast<const double*>(ws), partials);
        }
    }
    for (int i = 0; i < n; i += GRAD_TABLE) {
        const cudaError_t e = launch_any(list + i, std::min(n - i, GRAD_TABLE), true, given, ws, partials,
                                         given || i ? static_cast<float*>(nullptr) : norm, max_norm, num_sms,
                                         static_cast<int*>(nullptr), stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mmbwd
