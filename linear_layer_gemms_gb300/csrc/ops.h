// Internal declarations of the kernels other than the tensor-core kernel (the
// fp32 FFMA path, the fp32 tensor-core path's passes, the encoder and
// LayerNorm backwards), shared with the C-ABI layer. Not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mmbwd {

// Test hook (mmbwd_debug_fail_next_launch): true for the next n calls, set by
// the test; every launch function checks it before it enqueues anything and
// then fails as the runtime does when it refuses a launch, so the error path
// of each entry point can be exercised without a GPU fault.
bool take_injected_launch_failure();

// Test hook (mmbwd_debug_hold_stream): one thread that lets the next launch on the
// stream begin and stays for `ns`.
cudaError_t hold_launch(uint64_t ns, cudaStream_t stream);

// ------------------------------------------------------------ fp32 SIMT path
constexpr int SIMT_BM = 128;
constexpr int SIMT_BN = 128;
constexpr int SIMT_BK = 8;
constexpr int SIMT_THREADS = 256;

cudaError_t simt_launch(float* dinp, float* dweight, float* dbias, const float* dout,
                        const float* inp, const float* weight, int64_t BT, int64_t C, int64_t OC,
                        cudaStream_t stream);

// out (BT x OC) = inp (BT x C) . weight^T + bias (bias may be null), fp32 FFMA.
cudaError_t simt_forward_launch(float* out, const float* inp, const float* weight, const float* bias,
                                int64_t BT, int64_t C, int64_t OC, cudaStream_t stream);

// out[r, o] = bias[o], or 0 without a bias (the forward when C == 0).
cudaError_t fill_rows_launch(void* out, const void* bias, int64_t rows, int64_t cols, int dtype,
                             cudaStream_t stream);

// dbias = column sums of dout (used when C == 0, where no GEMM tile exists).
cudaError_t colsum_launch(void* dbias, const void* dout, int64_t BT, int64_t OC, int dtype, bool sr, uint64_t sr_seed,
                          cudaStream_t stream);

// ---------------------------------------------------------------- fp32 on the tensor cores (3xTF32)

// (no workspace: the kernel splits the raw fp32 operands in shared memory)
bool x3_shape_ok(int64_t BT, int64_t C, int64_t OC);
cudaError_t x3_launch(float* dinp, float* dweight, float* dbias, const float* dout, const float* inp,
                      const float* weight, int64_t BT, int64_t C, int64_t OC, int num_sms, cudaStream_t stream);
bool x3_forward_shape_ok(int64_t BT, int64_t C, int64_t OC);
cudaError_t x3_forward_launch(float* out, const float* inp, const float* weight, const float* bias, int64_t BT,
                              int64_t C, int64_t OC, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- encoder backward

size_t enc_workspace_bytes(int64_t BT, int64_t C);
size_t enc_plan_bytes(int64_t BT, int64_t C);           // the tables encbwd_prepare writes
size_t enc_run_workspace_bytes(int64_t BT, int64_t C);  // scratch of a planned run
cudaError_t enc_prepare_launch(void* plan, const int32_t* inp, int64_t B, int64_t T, int64_t C, int64_t V,
                               cudaStream_t stream);
cudaError_t enc_run_planned_launch(void* dwte, void* dwpe, const void* dout, void* plan, int64_t B, int64_t T,
                                   int64_t C, int64_t V, int dtype, void* ws, int num_sms, cudaStream_t stream,
                                   bool sr, uint64_t seed);
cudaError_t enc_launch(void* dwte, void* dwpe, const void* dout, const int32_t* inp, int64_t B, int64_t T, int64_t C,
                       int64_t V, int dtype, void* ws, int num_sms, cudaStream_t stream, bool sr = false,
                       uint64_t seed = 0);
cudaError_t enc_read_status(int* code, int* info3, bool reset);

// ---------------------------------------------------------------- LayerNorm backward

struct LnPlan {
    int wide = 0;            // 1: rows too wide for the fused kernel (row sums, then column tiles)
    int vpl = 0;             // 16-byte column vectors per thread and row
    int team_warps = 0;      // warps that share one row
    int warps = 0;           // warps per block
    int grid = 0;            // blocks (one per SM), each a contiguous range of rows
    int64_t rows_per_block = 0;
    size_t off_ring = 0;     // start of the teams' row buffers in shared memory
    size_t smem = 0;         // weight (fp32) + row-sum exchange + barriers + row buffers
    size_t ws_bytes = 0;     // per-block partial sums, fp32 [grid][2][C] (+ the row sums when wide)
    int col_tiles = 0;       // wide: column tiles of 256 vectors
};

int ln_vec_elems(int dtype);
cudaError_t ln_make_plan(int64_t BT, int C, int dtype, int num_sms, LnPlan* plan);
cudaError_t ln_launch(const LnPlan& plan, void* dinp, void* dweight, void* dbias, const void* dout,
                      const void* inp, const void* weight, const float* mean, const float* rstd, int64_t BT,
                      int C, int dtype, void* ws, cudaStream_t stream);
cudaError_t ln_read_status(int* code, int* info3, bool reset);

// ---------------------------------------------------------------- epilogues with an activation

// fp32 on the CUDA cores: out = act(inp . weight^T + bias) + residual, pre (may be null)
// the argument of act; dpre = (dout . weight) * act'(pre), dweight and dbias as in the
// backward. `tile`: 32 or 64.
cudaError_t simt_small_forward_launch(int tile, float* out, float* pre, const float* inp, const float* weight,
                                      const float* bias, const float* residual, int64_t BT, int64_t C, int64_t OC,
                                      int act, int num_sms, cudaStream_t stream);
cudaError_t simt_small_run_launch(int tile, float* dpre, float* dweight, float* dbias, const float* dout,
                                  const float* inp, const float* weight, const float* pre, int64_t BT, int64_t C,
                                  int64_t OC, int act, int num_sms, cudaStream_t stream);
// Which kernel takes these products in fp32.
enum class ActPath { TOKENS, SMALL_32, SMALL_64, SPANS };  // tokens_act.cu, the two above, tc_launch_span_*
ActPath act_forward_path(int64_t BT, int64_t C, int64_t OC, int num_sms);
ActPath act_run_path(int64_t BT, int64_t C, int64_t OC, int num_sms);
// The forward for few tokens: fp32 64 at most (ACT_TOKENS), bf16 by the time of either kernel.
constexpr int64_t ACT_TOKENS = 64;
bool tokens_act_takes_bf16(int64_t T, int64_t K, int64_t N, int num_sms);
cudaError_t tokens_act_launch(void* out, void* pre, const void* inp, const void* weight, const void* bias,
                              const void* residual, int64_t T, int64_t K, int64_t N, int act, int dtype, int num_sms,
                              cudaStream_t stream);
// dpre = dout * act'(pre), n values; pre is null without an activation
cudaError_t act_backward_launch(void* dpre, const void* dout, const void* pre, int64_t n, int act, int dtype,
                                cudaStream_t stream);
// the forward without a product (C == 0): pre = bias, out = act(bias) + residual
cudaError_t act_rows_launch(void* out, void* pre, const void* bias, const void* residual, int64_t rows, int64_t cols,
                            int act, int dtype, cudaStream_t stream);

// ---------------------------------------------------------------- norms around a block

struct ResidualNorm {
    // forward: out, residual_out, the statistics written; backward: the statistics read
    void *out = nullptr, *residual_out = nullptr;
    float *mean_post = nullptr, *rstd_post = nullptr, *mean = nullptr, *rstd = nullptr;
    const void *x = nullptr, *branch = nullptr, *gate = nullptr;
    const void *weight_post = nullptr, *bias_post = nullptr, *weight = nullptr, *bias = nullptr;
    // backward
    void *dx = nullptr, *dbranch = nullptr;
    void *dgate = nullptr, *dweight_post = nullptr, *dbias_post = nullptr, *dweight = nullptr, *dbias = nullptr;
    const void *dout = nullptr, *dresidual = nullptr, *residual = nullptr;
    float* ws = nullptr;
    int64_t rows = 0;
    int C = 0;
    float scale = 1.f, eps = 0.f;
    int post = 0, norm = 0;
};
cudaError_t residual_forward_launch(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream);
cudaError_t residual_backward_launch(const ResidualNorm& a, int dtype, int num_sms, cudaStream_t stream);
size_t residual_backward_workspace(int64_t rows, int64_t C, int dtype);

// ---------------------------------------------------------------- gradient norm and clipping

struct GradTensor {
    const void* grad;
    void* out;
    int64_t count;  // > 0
    bool bf16;
};
constexpr int GRAD_TABLE = 1024;       // tensors of one launch (28 KB of kernel parameters)
constexpr int GRAD_BLOCKS_PER_SM = 4;  // of the norm: as many of its 256-thread blocks as are resident
constexpr int GRAD_SCALE_BLOCKS_PER_SM = 8;
constexpr int GRAD_MAX_BLOCKS = 1536;  // partial sums of one launch
// given == nullptr: the norm of the list first, into `ws` and `norm`; `scale`: the outs.
cudaError_t grad_launch(const GradTensor* list, int n, float* norm, const float* given, bool scale, float max_norm,
                        double* ws, int num_sms, cudaStream_t stream);

}  // namespace mmbwd
