/*
 * grad_clip.h -- C ABI of the global gradient norm over many tensors, and of clipping
 * by it, in the same library (libmmbwd.so): the step between the backward and the
 * optimizer. Over all values g of all tensors of a list
 *
 *     norm = sqrt(sum g^2)
 *     coef = max_norm / (norm + 1e-6)  where that is below 1, else 1
 *     out  = coef * g
 *
 * The device keeps the norm; nothing is read back and the host does not wait. Squares
 * are summed in fp32 over at most 64 values and in 64 bits beyond, in a fixed order;
 * values whose squares leave the range of fp32 are summed scaled by a power of two, so
 * the norm is right for every finite input whose norm is an fp32 number. A list with
 * an infinity has norm inf (coef 0: its finite values become 0, the infinite ones
 * NaN); one with a NaN has norm NaN, and clipping makes every value NaN: a program
 * that skips such steps reads the norm first.
 */
#ifndef GRAD_CLIP_H
#define GRAD_CLIP_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "mmbwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of a list. Any count and any address that is a multiple of the element
 * size (16-byte vectors are used where both addresses allow it). */
typedef struct mmbwd_grad {
    void* grad;     /* device, `count` values */
    void* out;      /* device, where the clipped values go; NULL, or grad itself: in place */
    int64_t count;  /* 0: nothing, the pointers are not looked at */
    int64_t dtype;  /* MMBWD_F32 or MMBWD_BF16, of both; the types of a list may differ */
} mmbwd_grad;

/*
 * mmbwd_grad_norm -- enqueue norm = sqrt(sum g^2) over a list (outs are not looked at).
 *
 *   norm       device, one fp32, 4-byte aligned, written
 *   list       host, n entries, read before the call returns; a tensor may be in it twice
 *   workspace  device, 256-byte aligned, mmbwd_grad_workspace_bytes() bytes: the caller's,
 *              so that calls with workspaces of their own may overlap
 *
 * n == 0 gives norm 0. Returns MMBWD_OK or a negative MMBWD_ERR_* code with nothing
 * enqueued (ERR_ALIAS: norm or the workspace overlaps a tensor).
 */
int mmbwd_grad_norm(float* norm, const mmbwd_grad* list, int n, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/*
 * mmbwd_grad_clip -- enqueue the norm and out = coef * g. Tensors clipped in place are
 * not written where coef is 1. max_norm is finite and >= 0. ERR_ALIAS also where an
 * output overlaps another output or another tensor of the list.
 */
int mmbwd_grad_clip(float* norm, const mmbwd_grad* list, int n, float max_norm, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/*
 * mmbwd_grad_scale -- the second half of mmbwd_grad_clip with a norm that is already on
 * the device (one that several lists' norms were joined into, for example).
 */
int mmbwd_grad_scale(const mmbwd_grad* list, int n, const float* norm, float max_norm, cudaStream_t stream);

/* Bytes of workspace that a list of n tensors needs (0 for n < 0). */
size_t mmbwd_grad_workspace_bytes(int n);

#ifdef __cplusplus
}
#endif

#endif /* GRAD_CLIP_H */
