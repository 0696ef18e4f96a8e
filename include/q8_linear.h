/*
 * q8_linear.h -- C ABI of the 8-bit linear layer in the same library
 * (libmmbwd.so) as the linear-layer backward: quantisation in blocks of 128,
 * the forward product, and the backward that reads an 8-bit checkpoint of the
 * activations.
 *
 * The 8-bit form of a matrix X (rows x K, row-major). Each row is cut into
 * blocks of 128 consecutive values (the last one shorter). With amax the
 * largest finite |x| of a block and MAX the format's largest value (448 for
 * MMBWD_E4M3, 57344 for MMBWD_E5M2):
 *
 *     s = the smallest whole number >= -127 with amax <= MAX * 2^s
 *         (0 for a block without a nonzero finite value)
 *     q = x * 2^-s rounded once to the 8-bit format, to nearest even
 *
 * so no value saturates, and q * 2^s is exact in fp32 (but for values that round up to
 * 2^128, an infinity there) and, where s is at least -124 (E4M3) or -117 (E5M2), in bf16
 * too: below that the least values fall under bf16's smallest. The scale is a power of two: an 8-bit float keeps the same relative step at every
 * scale, so a finer scale would only move the range's lower end by part of a
 * binade. An infinity or a NaN becomes the format's NaN (it does not enter amax).
 *
 *   values  rows x ld bytes, ld = K rounded up to 16; bytes K .. ld-1 of a row
 *           are zero
 *   scales  one byte s + 127 per block; with G = ceil(ceil(K / 128) / 4) the byte of
 *           row r, block k is at
 *             ((r / 128) * G + k / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + k % 4
 *           (tiles of 128 rows x 4 blocks in the order the tensor cores take
 *           them); bytes of no row or block hold 127
 *
 * The "row form" of X is the 8-bit form of X itself; its "column form" is that
 * of X transposed (cols x rows values: blocks of 128 rows of one column). A
 * product contracts over the index that the blocks run along:
 *
 *   product                              reads
 *   out     = inp . weight^T  (over C)   inp row form,     weight row form
 *   dinp    = dout . weight   (over OC)  dout row form,    weight column form
 *   dweight = dout^T . inp    (over B*T) dout column form, inp column form
 *
 * The column form of inp is therefore all that the forward has to keep for
 * the backward: the activation checkpoint, half the bytes of a bf16 one.
 *
 * Element types: MMBWD_F32 / MMBWD_BF16 codes of mmbwd.h for the unquantised
 * tensors. Products of 8-bit values are exact; sums are formed in fp32 on the
 * tensor cores, each block's products times both blocks' scales; each output
 * element is rounded once. The tensor core cuts each accumulation of 32 products
 * toward zero: sums whose terms all have one sign come out low by a share that
 * grows with their length (measured 1e-7 at 1024 terms, 3e-6 at 8192, 4e-5 at
 * 51200); where signs mix it stays near 1e-7. Repeated calls give bitwise identical results (no
 * float atomics; every sum in an order fixed by shape and device).
 *
 * Every call enqueues on `stream` and returns MMBWD_OK or a negative
 * MMBWD_ERR_* code with nothing enqueued. No result depends on anything kept
 * between calls (the library remembers how it split a shape's work): what a call
 * needs beyond its tensors is a workspace of the caller's, so calls with their own
 * workspaces may overlap on different streams or in different captured graphs, from
 * one thread or several. The first call of a shape searches for the split on the host
 * (0.2 to 1 ms for a backward); calls of other threads do not wait for it.
 *
 * The waits inside the product kernels are bounded: by MMBWD_WAIT_TIMEOUT_NS
 * nanoseconds each, read from the environment at every call (2 s where it is not set), as
 * in the bf16 kernel. One that runs out leaves the call's outputs incomplete and is
 * reported by mmbwd_device_status.
 *
 * For tuning and tests the environment overrides the work split:
 * MMBWD_Q8_SPLITS = "<dinp>,<dweight>" (pieces of each product's reduction, 0: the
 * planner's choice) and MMBWD_Q8_TILE_N = "<dinp>,<dweight>" (tile widths, 128 or
 * 256; 0: the planner's) of the backward, whether a call wants one output or both;
 * the first width is the forward's too. MMBWD_Q8_TOKEN_SPLITS (1, 2, 4 or 8 CTAs to a
 * tile) of the forward for few tokens. The workspace size follows the first two. An
 * override that no work split can meet is dropped.
 */
#ifndef Q8_LINEAR_H
#define Q8_LINEAR_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "mmbwd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MMBWD_E4M3 0 /* 4 exponent bits, 3 mantissa bits, largest value 448 */
#define MMBWD_E5M2 1 /* 5 exponent bits, 2 mantissa bits, largest value 57344 */

#define MMBWD_Q8_BLOCK 128

/* mmbwd_q8_backward: add to the old contents instead of overwriting them */
#define MMBWD_Q8_ADD_DINP 1
#define MMBWD_Q8_ADD_DWEIGHT 2

/* Bytes of the values and of the scales of a rows x K matrix in 8-bit form (0
 * for invalid or empty sizes). */
size_t mmbwd_q8_data_bytes(int64_t rows, int64_t K);
size_t mmbwd_q8_scale_bytes(int64_t rows, int64_t K);

/*
 * mmbwd_q8_quantize -- enqueue the quantisation of x (rows x cols), read once.
 *
 *   q, scale       device, row form (rows x cols), written; both NULL: not wanted
 *   qt, scale_t    device, column form (cols x rows), written; both NULL: not wanted
 *   colsum_or_null device, (cols), type of x, overwritten with the sums of x over its
 *                  rows (of the unquantised values, fp32): dbias when x is dout
 *   x              device, (rows, cols), read only
 *   workspace      device, mmbwd_q8_quantize_workspace_bytes() bytes, 256-byte
 *                  aligned, contents ignored and overwritten; used with colsum of more
 *                  than 1024 rows (may be NULL where 0 bytes are needed)
 *   rows, cols     >= 0; cols times the element size a multiple of 16 bytes
 *   dtype          MMBWD_F32 or MMBWD_BF16 (x and colsum)
 *   format         MMBWD_E4M3 or MMBWD_E5M2 (both forms)
 *
 * Errors: ERR_DTYPE (dtype or format), ERR_SHAPE (a size negative or too large;
 * a workspace too small), ERR_NULL (a missing tensor, or one of a pair given
 * without the other), ERR_ALIGN (16 bytes; workspace 256), ERR_ALIAS (an output
 * overlaps anything else), ERR_MEMORY, ERR_ARCH, ERR_CUDA. rows == 0 sets colsum
 * to zero; cols == 0 enqueues nothing.
 */
int mmbwd_q8_quantize(void* q, void* scale, void* qt, void* scale_t, void* colsum_or_null, const void* x,
                      void* workspace, size_t workspace_bytes, int64_t rows, int64_t cols, int dtype, int format,
                      cudaStream_t stream);
size_t mmbwd_q8_quantize_workspace_bytes(int64_t rows, int64_t cols);

/*
 * mmbwd_q8_forward -- enqueue out (B*T, OC) = inp . weight^T + bias (overwritten).
 *
 *   out                     device, (B*T, OC), type `dtype`, written
 *   inp_q, inp_scale        device, row form of inp (B*T x C), format inp_format
 *   weight_q, weight_scale  device, row form of weight (OC x C), format weight_format
 *   bias_or_null            device, (OC), type `dtype`
 *
 * OC a multiple of 4; C and B*T any size. No
 * workspace. C == 0 gives out = bias (or 0); B*T == 0 or OC == 0 enqueue nothing.
 * Errors as mmbwd_q8_quantize.
 */
int mmbwd_q8_forward(void* out, const void* inp_q, const void* inp_scale, const void* weight_q,
                     const void* weight_scale, const void* bias_or_null, int64_t B, int64_t T, int64_t C, int64_t OC,
                     int inp_format, int weight_format, int dtype, cudaStream_t stream);

/*
 * mmbwd_q8_backward -- enqueue dinp (B*T, C) = dout . weight and
 * dweight (OC, C) = dout^T . inp, from 8-bit operands.
 *
 *   dinp_or_null      device, (B*T, C), type dinp_dtype, written; NULL: not wanted
 *                     (its operands dout_q, dout_scale, weight_qt, weight_scale_t
 *                     are then not read and may be NULL)
 *   dweight_or_null   device, (OC, C), type dweight_dtype, written; NULL: not wanted
 *                     (dout_qt, dout_scale_t, inp_qt, inp_scale_t may then be NULL)
 *   dout_q, dout_scale          row form of dout (B*T x OC), format dout_format
 *   dout_qt, dout_scale_t       column form of dout (OC x B*T), same format
 *   inp_qt, inp_scale_t         column form of inp (C x B*T): the forward's
 *                               checkpoint, format inp_format
 *   weight_qt, weight_scale_t   column form of weight (C x OC), format weight_format
 *   workspace         device, mmbwd_q8_backward_workspace_bytes() bytes, 256-byte
 *                     aligned, contents ignored and overwritten (may be NULL when 0)
 *   accumulate        MMBWD_Q8_ADD_DINP | MMBWD_Q8_ADD_DWEIGHT: add to the old
 *                     contents (one rounding after the addition); a clear bit overwrites
 *
 * dbias is the column sum that mmbwd_q8_quantize forms while it quantises dout.
 * C is a multiple of 4, OC and B*T any size. An empty sum
 * (OC == 0 for dinp, B*T == 0 for dweight) overwrites with zeros, or adds
 * nothing. Errors as mmbwd_q8_quantize; ERR_SHAPE also for unknown accumulate bits.
 */
int mmbwd_q8_backward(void* dinp_or_null, void* dweight_or_null, const void* dout_q, const void* dout_scale,
                      const void* dout_qt, const void* dout_scale_t, const void* inp_qt, const void* inp_scale_t,
                      const void* weight_qt, const void* weight_scale_t, void* workspace, size_t workspace_bytes,
                      int64_t B, int64_t T, int64_t C, int64_t OC, int dout_format, int inp_format, int weight_format,
                      int dinp_dtype, int dweight_dtype, int accumulate, cudaStream_t stream);
size_t mmbwd_q8_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t OC);

/* Test hook: how many times the library has searched for a work split of the products.
 * The outcome is remembered per shape (for about two thousand), so a shape seen
 * before is not searched for again, whatever the types and the accumulate bits. */
long long mmbwd_q8_debug_plan_searches(void);

/* Self-test of the bounded waits: one thread waits as the product kernel (kernel 0) or
 * the few-tokens kernel (1) does, on a barrier that nothing completes, and gives up
 * after timeout_ns (0: the limit the kernels take), two seconds at most. Synchronises
 * the device; the failure is then in the status word, for mmbwd_device_status to report and clear.
 * Returns a status of the launch (ERR_SHAPE: no such kernel). */
int mmbwd_q8_selftest_wait_timeout(int kernel, uint64_t timeout_ns);

#ifdef __cplusplus
}
#endif

#endif /* Q8_LINEAR_H */
