// Internal declarations of the 8-bit linear layer (quantisation, products) and
// of the LayerNorm forward, shared with the C-ABI layer. Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <cstdlib>

namespace mmbwd {

constexpr int Q8_BLOCK = 128;  // values per scale

// Blocks of a row of K values, groups of four blocks, bytes between rows.
inline int64_t q8_blocks(int64_t K) { return (K + Q8_BLOCK - 1) / Q8_BLOCK; }
inline int64_t q8_groups(int64_t K) { return (q8_blocks(K) + 3) / 4; }
inline int64_t q8_ld(int64_t K) { return (K + 15) & ~int64_t(15); }

// Column sums of at most this many row blocks are joined by the CTAs of one
// cluster, in the quantising kernel; more of them through a workspace and a second
// kernel (500 x 520: 4.1 us on the device against 4.0, 6.4 us of host time against 8.1).
constexpr int64_t Q8_SUM_CLUSTER = 8;

// q/scale and qt/scale_t: either pair may be null. `partials` holds
// ceil(rows / 128) * cols floats when colsum is wanted of more than
// Q8_SUM_CLUSTER row blocks.
cudaError_t q8_quantize_launch(uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* colsum, const void* x,
                               float* partials, int64_t rows, int64_t cols, int dtype, int format,
                               cudaStream_t stream);

// One product D (M x N, row-major, leading dimension N) = A (M x K) . B (N x K)^T
// (+ bias per column, + the old D), A and B in 8-bit form.
struct Q8Product {
    void* D = nullptr;
    const void* bias = nullptr;  // per column of D, type of D; null: none
    const uint8_t *A = nullptr, *a_scale = nullptr, *B = nullptr, *b_scale = nullptr;
    int64_t M = 0, N = 0, K = 0;
    int a_format = 0, b_format = 0;
    int dtype = 0;  // of D and bias
    int add = 0;    // add to the old D
    int slot = 0;   // which value of an override is its: 0 the first (dinp, the forward), 1 the second (dweight)
};

// One or two products in one launch (their K ranges split where that fills the
// device and `may_split`; the split sums then need the workspace). The
// workspace depends on the shapes only.
size_t q8_products_workspace(const Q8Product* products, int n, int num_sms);
cudaError_t q8_products_launch(const Q8Product* products, int n, bool may_split, void* ws, size_t ws_bytes, int num_sms,
                               cudaStream_t stream);
// How many times a shape's tile widths and splits have been searched for.
long long q8_plan_searches();
// Whether the forward takes the few-tokens kernel: always up to 64 tokens, and
// up to 256 while its 128 x 64 tiles are at most half the SMs, so that several
// CTAs share each tile's K. Measured (us, this kernel against the pair kernel): 1 token
// 1600 -> 4800 5.2 / 7.3; 64 tokens 6.9 / 7.4; 64 x 768 -> 768 4.5 / 4.5; 128 x 6400 ->
// 1600 9.1 / 18.1; 128 x 12800 -> 4096 22.8 / 32.8; 256 x 6400 -> 1600 12.8 / 18.2;
// beyond the rule 192 x 12800 -> 4096 36.8 / 32.8, 192 x 1600 -> 4800 8.0 / 7.7.
inline bool q8_few_tokens(int64_t tokens, int64_t N, int num_sms) {
    return tokens <= 64 || (tokens <= 256 && (tokens + 63) / 64 * ((N + 127) / 128) <= num_sms / 2);
}

// The forward (D overwritten) for few tokens (rows of A).
cudaError_t q8_tokens_launch(const Q8Product& product, int num_sms, cudaStream_t stream);
cudaError_t q8_tokens_read_status(int* code, int* info3, bool reset);
cudaError_t q8_read_status(int* code, int* info3, bool reset);

// How long a wait of the two product kernels may last: MMBWD_WAIT_TIMEOUT_NS, as
// for the bf16 kernel, else 2 s.
inline unsigned long long q8_wait_limit_ns() {
    const char* s = std::getenv("MMBWD_WAIT_TIMEOUT_NS");
    char* end = nullptr;
    const long long v = s && *s ? std::strtoll(s, &end, 10) : 0;
    return v > 0 && *end == '\0' ? static_cast<unsigned long long>(v) : 2000000000ull;
}
cudaError_t q8_selftest_wait(unsigned long long limit_ns);
cudaError_t q8_tokens_selftest_wait(unsigned long long limit_ns);

cudaError_t ln_forward_launch(void* out, float* mean, float* rstd, const void* inp, const void* weight,
                              const void* bias, int64_t BT, int C, float eps, int dtype, int num_sms,
                              cudaStream_t stream);

}  // namespace mmbwd
