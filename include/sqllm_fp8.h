/*
 * sqllm_fp8.h -- C ABI of 8-bit floating point weights with a scale for each
 * block of 128 columns, on AMD Instinct MI355X (gfx950): the quantiser and
 * the product, for matrices that are not kept as lookup tables and for
 * batches above the 16 of sqllm.h.
 *
 * Stored form of a matrix of `cols` columns (weights, and activations inside
 * the product): per row and block of 128 columns an integer s, the smallest
 * with max |v| <= 448 * 2^s over the block, and per value the e4m3 number
 * (OCP FP8 E4M3: 4 exponent bits, 3 mantissa bits, largest value 448, no
 * infinities) nearest to v * 2^-s, ties to even.  A power of two scales
 * without rounding, and the matrix cores take it as an operand, so it costs
 * the product nothing.
 *   q      uint8 [rows][sqllm_fp8_cols(cols)]: the e4m3 codes, columns
 *          beyond `cols` zero; 16-byte aligned
 *   scale  uint8 [rows][sqllm_fp8_scale_pitch(cols)]: s + 127 per block,
 *          127 beyond the last block; 4-byte aligned
 * A block of zeros has s = 0.  Infinities and NaN take no part in s and are
 * stored as NaN (a block of nothing else has s = 0).
 *
 * Conventions are those of sqllm.h (device pointers, fp16 as bit patterns,
 * asynchronous on `stream`, argument errors on the host before any launch),
 * except that the product's workspace is plain scratch, 256-byte aligned: it
 * need not be zero, holds nothing between calls and is left with any
 * contents, so it must not be given to the calls of sqllm.h.
 */
#ifndef SQLLM_FP8_H
#define SQLLM_FP8_H

#include "sqllm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns of q (cols rounded up to 128) and bytes of a row of scales (one
 * per block, rounded up to 4); 0 for cols outside [1, 2^24]. */
int64_t sqllm_fp8_cols(int64_t cols);
int64_t sqllm_fp8_scale_pitch(int64_t cols);

/*
 * sqllm_fp8_quantize -- fp16 values to the stored form.
 *   x: fp16, row r at x + r * ldx (ldx >= cols, in values), 2-byte aligned;
 *   rows >= 1, 1 <= cols <= 2^24, rows * scale pitch <= 2^30 - 256 (else
 *   SQLLM_ERR_SHAPE).
 */
sqllm_status sqllm_fp8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, uint8_t *q,
                                uint8_t *scale, hipStream_t stream);

/* Scratch bytes of the product of x in fp16, with room for its rounded form,
 * and of x in the stored form: 256 where no columns are split.  0 if the sizes
 * are out of range. */
size_t sqllm_fp8_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);
size_t sqllm_fp8_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);

/*
 * sqllm_fp8_gemm -- y = x W^T with W [rows][cols] in the stored form and x
 * fp16 [batch][cols], which the call rounds to the stored form first.
 *   y[b][r] = sum over blocks 2^(sx + sw) * sum_c qx[b][c] * qw[r][c]
 * Sums in fp32, in a fixed order (repeated calls give identical bits), one
 * rounding to fp16.  The matrix cores add the products of each eight
 * adjacent columns on a grid 13 bits below the largest of them before the
 * fp32 sum: with activations as in a decoder about 2^-14 of y, a quarter of
 * its own rounding.  A value of x that is infinite or NaN makes its row of y
 * NaN.
 *   x: 2-byte aligned, contiguous; y: fp16 [batch][rows], 2-byte aligned,
 *   must not overlap an input.  The bounds of sqllm_fp8_quantize hold for both
 *   matrices (else SQLLM_ERR_BATCH for x) and rows * batch <= 2^38 (else
 *   SQLLM_ERR_SHAPE).
 */
sqllm_status sqllm_fp8_gemm(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols, const uint16_t *x,
                            int64_t batch, uint16_t *y, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * sqllm_fp8_gemm_stored -- the same with x already in the stored form, as
 * sqllm_fp8_quantize and sqllm_rms_norm_fp8 leave it: xq uint8 [batch]
 * [sqllm_fp8_cols(cols)], 16-byte aligned, xscale uint8 [batch]
 * [sqllm_fp8_scale_pitch(cols)], 4-byte aligned; scratch of
 * sqllm_fp8_stored_workspace_bytes.
 */
sqllm_status sqllm_fp8_gemm_stored(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                   const uint8_t *xq, const uint8_t *xscale, int64_t batch, uint16_t *y,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SQLLM_FP8_H */
