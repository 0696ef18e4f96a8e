/*
 * layernorm_forward.h -- C ABI of the GPT-2 LayerNorm forward in the same
 * library (libmmbwd.so), with the row statistics that lnbwd_run
 * (layernorm_backward.h) reads. For every row of BT = B*T rows of width C
 *
 *     mean = (1/C) sum_i x_i,   var = (1/C) sum_i (x_i - mean)^2,
 *     rstd = 1 / sqrt(var + eps),
 *     out_i = (x_i - mean) * rstd * weight_i + bias_i
 *
 * Sums are formed in fp32 from the row held on chip (the variance from the
 * differences, not from the squares); the mean of a sum that is exact is exact, so
 * that a row of one value gives the bias; out is rounded once. Rows are
 * independent and each row's sums run in a fixed order: repeated calls give
 * bitwise identical results.
 */
#ifndef LAYERNORM_FORWARD_H
#define LAYERNORM_FORWARD_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "mmbwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest C accepted (as the backward's). */
#define LNFWD_MAX_C (1 << 20)

/*
 * lnbwd_forward -- enqueue the LayerNorm forward of B*T rows of width C.
 *
 *   out           device, (B*T, C), written
 *   mean_or_null  device, (B*T) fp32, written (NULL: not wanted)
 *   rstd_or_null  device, (B*T) fp32, written (NULL: not wanted)
 *   inp           device, (B*T, C), read only; may be `out` itself (in place)
 *   weight, bias_or_null  device, (C), read only; a NULL bias is zero
 *   eps           added to the variance; finite and >= 0 (GPT-2: 1e-5)
 *   dtype         MMBWD_F32 or MMBWD_BF16 (out, inp, weight, bias)
 *
 * C times the element size a multiple of 16 bytes, out, inp, weight and bias
 * 16-byte aligned, mean and rstd 4-byte aligned. Returns MMBWD_OK or a negative
 * MMBWD_ERR_* code with nothing enqueued (ERR_SHAPE: a size or eps out of
 * range; ERR_ALIAS: an output overlaps another tensor, unless out == inp). No
 * workspace. B*T == 0 or C == 0 enqueue nothing.
 */
int lnbwd_forward(void* out, float* mean_or_null, float* rstd_or_null, const void* inp, const void* weight,
                  const void* bias_or_null, int64_t B, int64_t T, int64_t C, float eps, int dtype,
                  cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYERNORM_FORWARD_H */
