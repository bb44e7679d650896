/*
 * sqllm_norm.h -- C ABI of the root-mean-square norm in front of a decoder's
 * products, on AMD Instinct MI355X (gfx950): with the residual's addition, its
 * output in fp16 or already in the 8-bit form that a product takes.
 *
 *   sum[r][c] = x[r][c] + residual[r][c], rounded to fp16 (x without residual)
 *   y[r][c]   = sum[r][c] / sqrt(mean over c of sum[r][c]^2 + eps) * weight[c]
 *
 * sum is the residual of the next addition, and the norm is that of the rounded
 * values: the same bits whether the addition was made here or before.  Squares
 * are exact, summed by eights in fp32 and further in fp64, in a fixed order; y
 * is computed in fp32 and rounded to the form that the call writes:
 *   sqllm_rms_norm       fp16 [rows][cols]
 *   sqllm_rms_norm_int8  the stored form of sqllm_int8.h (its integers without
 *                        rounding before: the root falls out of them)
 *   sqllm_rms_norm_fp8   the stored form of sqllm_fp8.h
 * A row of zeros with eps = 0 is 0 / 0: NaN.  An infinity in a row of sums
 * makes its own place NaN and the other values 0; a NaN makes the row NaN.
 *
 *   x, residual: fp16, row r at x + r * ldx, residual + r * ldr (>= cols, in
 *     values), 2-byte aligned; residual may be NULL, and sum with it
 *   weight: fp16 [cols], 2-byte aligned
 *   sum: fp16 [rows][cols], 2-byte aligned; NULL where it is not wanted.  It may
 *     be x or residual itself where that is contiguous; no output may overlap
 *     an input in any other way
 *   1 <= rows <= 2^30; 1 <= cols <= 2^24, for the 8-bit forms as they bound it;
 *   eps finite, >= 0 (else SQLLM_ERR_SHAPE)
 *
 * Conventions are those of sqllm.h (device pointers, fp16 as bit patterns,
 * asynchronous on `stream`, argument errors on the host before any launch).
 * No workspace.
 */
#ifndef SQLLM_NORM_H
#define SQLLM_NORM_H

#include "sqllm.h"

#ifdef __cplusplus
extern "C" {
#endif

sqllm_status sqllm_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                            const uint16_t *weight, int64_t rows, int64_t cols, float eps, uint16_t *sum, uint16_t *y,
                            hipStream_t stream);

/* q, scale: sqllm_int8.h; cols <= 131071. */
sqllm_status sqllm_rms_norm_int8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                 const uint16_t *weight, int64_t rows, int64_t cols, float eps, uint16_t *sum,
                                 int8_t *q, float *scale, hipStream_t stream);

/* q, scale: sqllm_fp8.h; rows * scale pitch <= 2^30 - 256. */
sqllm_status sqllm_rms_norm_fp8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                const uint16_t *weight, int64_t rows, int64_t cols, float eps, uint16_t *sum,
                                uint8_t *q, uint8_t *scale, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SQLLM_NORM_H */
