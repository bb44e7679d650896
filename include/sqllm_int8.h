/*
 * sqllm_int8.h -- C ABI of products in 8-bit integers with a scale for each
 * token and each channel, on AMD Instinct MI355X (gfx950): the quantiser, the
 * product, and the gated half of a feed-forward block (gate and up, the
 * activation and their product) in one call.  For weights kept as 8-bit
 * integers with a scale for each output channel, at any batch.
 *
 * Stored form of a matrix of `cols` columns (weights, and activations inside
 * the products): per row the scale max |v| / 127 over the row in fp32, and per
 * value the integer nearest to v * 127 / max |v|, ties to even.
 *   q      int8 [rows][sqllm_int8_cols(cols)]: the integers, columns beyond
 *          `cols` zero; 16-byte aligned
 *   scale  fp32 [rows]; 4-byte aligned
 * A row of zeros has scale 0.  A row that holds an infinity or a NaN has the
 * scale NaN and zeros: products with it are NaN.  Codes and scales made
 * elsewhere serve as well; -128 is a code like the others.
 *
 * Conventions are those of sqllm.h (device pointers, fp16 as bit patterns,
 * asynchronous on `stream`, argument errors on the host before any launch),
 * except that the products' workspace is plain scratch, 256-byte aligned: it
 * need not be zero, holds nothing between calls and is left with any
 * contents, so it must not be given to the calls of sqllm.h.
 */
#ifndef SQLLM_INT8_H
#define SQLLM_INT8_H

#include "sqllm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns of q: cols rounded up to 128; 0 for cols outside [1, 131071] (the
 * longest row whose sums of products fit 32 bits). */
int64_t sqllm_int8_cols(int64_t cols);

/*
 * sqllm_int8_quantize -- fp16 values to the stored form.
 *   x: fp16, row r at x + r * ldx (ldx >= cols, in values), 2-byte aligned;
 *   1 <= rows <= 2^30 (else SQLLM_ERR_SHAPE).
 */
sqllm_status sqllm_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, float *scale,
                                 hipStream_t stream);

/* Scratch bytes of the product, and of sqllm_int8_glu with two matrices of
 * that size; 0 if the sizes are out of range.  The first two are for x in
 * fp16, with room for its rounded form; with x in the stored form the calls
 * ask for no more than the other two, 256 bytes where no columns are split. */
size_t sqllm_int8_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);
size_t sqllm_int8_glu_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);
size_t sqllm_int8_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);
size_t sqllm_int8_glu_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);

/*
 * sqllm_int8_gemm -- y = x W^T with W [rows][cols] in the stored form.
 *   y[b][r] = xscale[b] * scale[r] * sum_c qx[b][c] * q[r][c]
 * The sum is exact; its conversion to fp32, the product of the two scales and
 * the product with it are rounded in fp32, and the result once to fp16.  So
 * the result does not depend on how the work is split.
 *   x, xscale: activations [batch][cols].  With xscale, x is int8 codes in the
 *     stored form (as sqllm_int8_quantize and sqllm_rms_norm_int8 leave them),
 *     16-byte aligned, and xscale fp32 [batch].  With xscale NULL, x is fp16,
 *     2-byte aligned, contiguous, which the call rounds to the stored form.
 *   y: fp16 [batch][rows], 2-byte aligned, must not overlap an input.
 *   1 <= rows, batch <= 2^28 (else SQLLM_ERR_SHAPE, SQLLM_ERR_BATCH) and
 *   rows * batch <= 2^38 (else SQLLM_ERR_SHAPE).
 */
sqllm_status sqllm_int8_gemm(const int8_t *q, const float *scale, int64_t rows, int64_t cols, const void *x,
                             const float *xscale, int64_t batch, uint16_t *y, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

/*
 * sqllm_int8_glu -- h = silu(x G^T) * (x U^T), silu(g) = g / (1 + e^-g), with
 * the matrices G (gate) and U (up), both [rows][cols] in the stored form.  The
 * two products are as sqllm_int8_gemm's before its rounding to fp16, silu and
 * the product in fp32, one rounding to fp16.  The other arguments and bounds
 * are sqllm_int8_gemm's; h is fp16 [batch][rows].
 */
sqllm_status sqllm_int8_glu(const int8_t *gate, const float *gate_scale, const int8_t *up, const float *up_scale,
                            int64_t rows, int64_t cols, const void *x, const float *xscale, int64_t batch, uint16_t *h,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Test-only export (not part of the stable contract).  sqllm_test_int8_plan:
 * how sqllm_int8_gemm (gated: sqllm_int8_glu) would compute a product of these
 * sizes, x in fp16 or (stored) in integers, without a device.  plan: HOST array
 * of 5 ints:
 *   plan[0]  1 if the quantiser's launch comes first
 *   plan[1]  the form: 0 streaming in the vector units, 1 streaming on the
 *            matrix cores, 2 tiles
 *   plan[2]  rows of x the kernel holds (1, 2, 4); blocks of 128 columns a wave
 *            (2, 4, 8, 16); the tile's number, 0 (256x256) to 10 (64x64 in three
 *            groups of waves)
 *   plan[3]  chunks of 1024 columns a wave (1 to 3); 0; splits of the columns
 *   plan[4]  0; 0; whole 256x256 tiles in front of the halves (0: no halves)
 */
sqllm_status sqllm_test_int8_plan(int64_t rows, int64_t cols, int64_t batch, int gated, int stored, int *plan);

#ifdef __cplusplus
}
#endif

#endif /* SQLLM_INT8_H */
