/*
 * residual_norm.h -- C ABI of the step between two blocks of a transformer in the same
 * library (libmmbwd.so): the norm after a block, its gate and scale, the sum with the
 * residual stream, and the norm before the next block, in one pass over the rows.
 * For every row of B*T rows of width C
 *
 *     residual_out = x + scale * gate * post(branch)
 *     out          = norm(residual_out)
 *
 * where post and norm are each one of
 *
 *     NONE    the row itself (norm == NONE: out is not computed)
 *     LAYER   (v - mean) * rstd * weight + bias,  var = (1/C) sum (v_i - mean)^2
 *     RMS     v * rstd * weight,                  var = (1/C) sum v_i^2
 *
 * with rstd = 1 / sqrt(var + eps), and gate is one value per channel (NULL: 1). A
 * GPT-2 block is post = NONE, norm = LAYER, no gate, scale 1; scale scales a
 * residual branch by depth; post and gate are those of blocks with a norm after
 * them or with a learned gate.
 *
 * All of it is fp32 from the row held on chip, each output rounded once: out is
 * formed from the fp32 residual_out, not from the rounded one. Sums run in a fixed
 * order: repeated calls give bitwise identical results.
 */
#ifndef RESIDUAL_NORM_H
#define RESIDUAL_NORM_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "mmbwd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LNBWD_NORM_NONE 0
#define LNBWD_NORM_LAYER 1
#define LNBWD_NORM_RMS 2

/* Largest C accepted: the widest row that a block's registers hold. */
#define LNBWD_RESIDUAL_MAX_C 32768

/*
 * lnbwd_residual_forward -- enqueue the forward of B*T rows.
 *
 *   out            device, (B*T, C), written; not used with norm == NONE
 *   residual_out   device, (B*T, C), written; may be `x` itself (in place)
 *   mean_post, rstd_post, mean, rstd
 *                  device, (B*T) fp32 each, written: the statistics that the backward
 *                  reads. NULL: not wanted; not used where the norm has none (mean of
 *                  an RMS norm, all of NONE)
 *   x, branch      device, (B*T, C), read only
 *   gate_or_null   device, (C), read only
 *   weight_post, bias_post_or_null
 *                  device, (C), read only: post's; weight required unless post is
 *                  NONE, the bias used with LAYER only
 *   weight, bias_or_null   likewise norm's
 *   scale          finite
 *   eps            of both norms; finite and >= 0
 *   post, norm     LNBWD_NORM_*
 *   dtype          MMBWD_F32 or MMBWD_BF16 (all but the statistics)
 *
 * C times the element size a multiple of 16 bytes, the statistics 4-byte and all
 * other pointers 16-byte aligned. Pointers that are not used are not looked at.
 * Returns MMBWD_OK or a negative MMBWD_ERR_* code with nothing enqueued (ERR_SHAPE:
 * a size, scale, eps, post or norm out of range; ERR_ALIAS: an output overlaps
 * another tensor, unless residual_out == x). No workspace. B*T == 0 or C == 0 enqueue
 * nothing.
 */
int lnbwd_residual_forward(void* out, void* residual_out, float* mean_post_or_null, float* rstd_post_or_null,
                           float* mean_or_null, float* rstd_or_null, const void* x, const void* branch,
                           const void* gate_or_null, const void* weight_post, const void* bias_post_or_null,
                           const void* weight, const void* bias_or_null, int64_t B, int64_t T, int64_t C, float scale,
                           float eps, int post, int norm, int dtype, cudaStream_t stream);

/*
 * lnbwd_residual_backward -- enqueue the gradients. With r = residual_out as stored,
 * n = (r - mean) * rstd, z = (branch - mean_post) * rstd_post (the row itself for
 * NONE, no mean for RMS) and g = weight * dout,
 *
 *     dx      = dresidual + rstd * (g - mean(g) - n * mean(g * n))    LAYER
 *               dresidual + rstd * (g - n * mean(g * n))              RMS
 *               dresidual                                             NONE
 *     dpost   = scale * gate * dx                     the gradient of post(branch)
 *     dbranch = dpost through post, likewise
 *     dgate        += sum over rows of scale * dx * post(branch)
 *     dweight_post += sum of dpost * z,   dbias_post += sum of dpost
 *     dweight      += sum of dout * n,    dbias      += sum of dout
 *
 *   dx                 device, (B*T, C), written: the gradient of x; may be
 *                      `dresidual` itself
 *   dbranch_or_null    device, (B*T, C), written (NULL: not wanted, as where it is
 *                      dx: post NONE, no gate, scale 1)
 *   dgate, dweight_post, dbias_post, dweight, dbias
 *                      device, (C), read and written (+=); NULL: not wanted. Not used
 *                      where there is no such parameter (dgate without a gate, the
 *                      biases of an RMS norm, all of NONE)
 *   dout               device, (B*T, C), read only; not used with norm == NONE
 *   dresidual_or_null  device, (B*T, C), read only: the gradient of residual_out
 *                      from where else it is used; NULL: none (not with norm == NONE)
 *   residual           device, (B*T, C), read only: the forward's residual_out; not
 *                      used with norm == NONE
 *   branch             device, (B*T, C), read only; not used (may be NULL) where neither post
 *                      nor dgate needs it
 *   gate_or_null, weight_post, bias_post_or_null, weight
 *                      device, (C), read only (bias_post for dgate alone)
 *   mean_post, rstd_post, mean, rstd
 *                      device, (B*T) fp32, read only: the forward's, those that the
 *                      norms have
 *   workspace          device, 256-byte aligned, lnbwd_residual_backward_workspace_bytes()
 *                      bytes: the caller's, so that calls with workspaces of their own
 *                      may overlap. Nothing in it is kept from call to call.
 *
 * Alignment, sizes and codes as the forward. B*T == 0 or C == 0 enqueue nothing. Sums
 * over rows are fp32 in a fixed order; each gradient is rounded once.
 */
int lnbwd_residual_backward(void* dx, void* dbranch_or_null, void* dgate_or_null, void* dweight_post_or_null,
                            void* dbias_post_or_null, void* dweight_or_null, void* dbias_or_null, const void* dout,
                            const void* dresidual_or_null, const void* residual, const void* branch,
                            const void* gate_or_null, const void* weight_post, const void* bias_post_or_null,
                            const void* weight, const float* mean_post, const float* rstd_post, const float* mean,
                            const float* rstd, void* workspace, size_t workspace_bytes, int64_t B, int64_t T, int64_t C,
                            float scale, int post, int norm, int dtype, cudaStream_t stream);

/* Bytes of workspace that lnbwd_residual_backward needs for these sizes, whatever its
 * other arguments (0 for invalid sizes and for none to do). */
size_t lnbwd_residual_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* RESIDUAL_NORM_H */
