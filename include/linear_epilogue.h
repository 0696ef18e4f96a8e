/*
 * linear_epilogue.h -- C ABI of the linear layer with an activation and a residual
 * in its epilogue, and of the gradients through the activation, in the same library
 * (libmmbwd.so). With BT = B*T and every tensor row-major and contiguous,
 *
 *     s   = inp (BT,C) . weight (OC,C)^T + bias
 *     pre = s                                   (kept for the backward, if wanted)
 *     out = act(s) + residual
 *
 * and, for a layer whose input inp = act(pre) is the activation of the layer before,
 *
 *     dpre     = (dout (BT,OC) . weight) * act'(pre)       (BT,C), overwritten
 *     dweight += dout^T . inp                               (OC,C)
 *     dbias    = sum over (b,t) of dout                     (OC), overwritten
 *
 * so that a GPT-2 MLP is two calls forward (fc with GELU keeping pre, projection with
 * the residual) and two calls backward (mmbwd_run_act for the projection, whose dpre
 * is the dout that mmbwd_run takes for fc).
 *
 * Sums, the bias, the activation and its derivative are fp32; each output is rounded
 * once (out from the fp32 sum, not from the rounded pre). bf16 products run on the
 * tensor cores. fp32 products are fp32 fused multiply-adds, or three tf32 products whose
 * accumulators are read back and added up in registers every 128 values of the
 * reduction (mmbwd_run's are not: the tensor core rounds toward zero). Relative errors of
 * those sums (2-norm, random operands): 6.3e-7 at 1600 values, 6.6e-7 at 9000, 8.5e-7 at
 * 65,536, 1.3e-6 at 262,144 and 2.4e-6 at 1,048,576, where the roundings of the running fp32 sum
 * are all there is; fused multiply-adds have 1.2e-7, 2.3e-7, 5.8e-7, 1.2e-6 and 2.3e-6. An
 * infinite fp32 operand may give NaN where the sum is infinite (infinity has no remainder
 * to split off), in the outputs that it belongs to.
 * MMBWD_ACT_F32_PATH in the environment forces the fp32 kernel: "32", "64" (tiles of
 * fused multiply-adds) or "spans"; MMBWD_ACT_BF16_PATH that of the bf16 forward: "tokens" (the
 * kernel for few tokens) or "tiles" (the tensor cores').
 */
#ifndef LINEAR_EPILOGUE_H
#define LINEAR_EPILOGUE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "mmbwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. */
#define MMBWD_ACT_NONE 0 /* act(x) = x */
#define MMBWD_ACT_GELU 1 /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))), GPT-2's */
#define MMBWD_ACT_SILU 2 /* x / (1 + exp(-x)) */
#define MMBWD_ACT_RELU 3 /* x if x > 0, else 0; its derivative at 0 is 0 */
/* A NaN stays a NaN in all of them, and in all derivatives but NONE's (1, whatever pre
 * holds). GELU and SILU of -inf are NaN (inf times 0), their derivatives at infinities the
 * limits 0 and 1. */

/*
 * mmbwd_forward_act -- enqueue the forward.
 *
 *   out               device, (BT, OC), written
 *   pre_or_null       device, (BT, OC), written (NULL: not wanted)
 *   inp               device, (BT, C),  read only
 *   weight            device, (OC, C),  read only
 *   bias_or_null      device, (OC),     read only; NULL: no bias
 *   residual_or_null  device, (BT, OC), read only; NULL: none; may be `out` itself
 *                     (the residual stream updated in place)
 *   act               MMBWD_ACT_*
 *   dtype             MMBWD_F32 or MMBWD_BF16 (all tensors)
 *
 * Alignment, sizes and status codes as mmbwd_forward (ERR_SHAPE also for an unknown
 * act and for OC > 8,388,480; ERR_ALIAS: out or pre overlaps another tensor, unless
 * out == residual). No workspace. C == 0 gives pre = bias (or 0).
 */
int mmbwd_forward_act(void* out, void* pre_or_null, const void* inp, const void* weight, const void* bias_or_null,
                      const void* residual_or_null, int64_t B, int64_t T, int64_t C, int64_t OC, int act, int dtype,
                      cudaStream_t stream);

/*
 * mmbwd_run_act -- enqueue the backward of a layer whose input is an activation.
 *
 *   dpre          device, (BT, C),  written (=); may be `pre` itself
 *   dweight       device, (OC, C),  read and written (+=)
 *   dbias_or_null device, (OC),     written (=); NULL skips it
 *   dout          device, (BT, OC), read only
 *   inp           device, (BT, C),  read only: act(pre), the layer's input
 *   weight        device, (OC, C),  read only
 *   pre           device, (BT, C),  read only (unless dpre is it); not used with
 *                 MMBWD_ACT_NONE (may be NULL)
 *   workspace     device, 256-byte aligned, mmbwd_run_act_workspace_bytes() bytes (NULL
 *                 where that is 0): the caller's, so that calls with workspaces of their own
 *                 may overlap. Nothing in it is kept from call to call.
 *
 * act = MMBWD_ACT_NONE is mmbwd_run with dinp overwritten. Otherwise as mmbwd_run:
 * B*T == 0 sets dbias to 0; OC == 0 sets dpre to 0 (the empty sum); C == 0 still computes dbias.
 */
int mmbwd_run_act(void* dpre, void* dweight, void* dbias_or_null, const void* dout, const void* inp,
                  const void* weight, const void* pre, void* workspace, size_t workspace_bytes, int64_t B, int64_t T,
                  int64_t C, int64_t OC, int act, int dtype, cudaStream_t stream);

/* Bytes of workspace mmbwd_run_act needs for this shape on the current device (a
 * full GB300 without a usable one); 0 when it needs none, and for invalid arguments. */
size_t mmbwd_run_act_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t OC, int dtype);

/*
 * mmbwd_act_backward -- enqueue dpre = dout * act'(pre), element by element, for an
 * activation that no product of this library's backward precedes (mmbwd_run_act has
 * it in its epilogue otherwise): the gradient through mmbwd_forward_act's activation,
 * after which mmbwd_run gives the layer's gradients and dout is the residual's.
 *
 *   dpre   device, n values, written; may be dout or pre itself
 *   dout   device, n values, read only
 *   pre    device, n values, read only; not used with MMBWD_ACT_NONE (may be NULL), which
 *          copies dout
 *
 * n >= 0, any; pointers 16-byte aligned.
 */
int mmbwd_act_backward(void* dpre, const void* dout, const void* pre, int64_t n, int act, int dtype,
                       cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_EPILOGUE_H */
