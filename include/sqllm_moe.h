/*
 * sqllm_moe.h -- C ABI of a mixture-of-experts layer for a few tokens, its
 * experts stored as dense-and-sparse LUT matrices (sqllm.h), on AMD Instinct
 * MI355X (gfx950).
 *
 *   l[t][e]  = sum_h x[t][h] * router[e][h]
 *   s[t][e]  = softmax over e of l[t][.], or 1 / (1 + exp(-l[t][e]))
 *   ids[t]   = the topk experts of the largest s[t][e] + bias[e], in
 *              descending order, ties to the lowest expert
 *   w[t][k]  = scale * s[t][ids[t][k]], divided by the sum over the topk
 *   a[t][k]  = silu(gate_e x_t) * (up_e x_t),  e = ids[t][k],
 *              silu(v) = v / (1 + exp(-v))
 *   y[t]     = sum_k w[t][k] * down_e a[t][k]
 *
 * gate_e and up_e are [inter][hidden], down_e is [hidden][inter]; each is
 * D + S of sqllm.h: packed 2-, 3- or 4-bit codes with a table of fp16
 * centroids per row, plus CSR outliers.  Which experts are read is decided
 * on the device; each one in use is read once, whatever tokens chose it.
 *
 * Arithmetic: router sums, scores and the comparison in 64 bits, so that the
 * choice does not depend on the order of a sum.  Expert products of two fp16
 * values are summed in fp32; a is stored as an unevaluated sum of two fp16
 * values, hi + lo * 2^-11, the form in which the matrix cores take it: 22
 * bits, or 2^-36 where |a| < 2^-14, and infinite from 65520 on, as an fp16
 * activation would be; y is rounded once.  Sums are taken in a fixed order:
 * repeated calls give identical bits.
 *
 * Shapes: 1 <= batch <= 16; 1 <= experts <= 512; 1 <= topk <= min(8,
 * experts); hidden and inter multiples of 256 in [256, 65536]; experts *
 * max(hidden, inter) < 2^30 (else SQLLM_ERR_BATCH for the batch,
 * SQLLM_ERR_SHAPE for the rest).
 *
 * Conventions are those of sqllm.h (device pointers, fp16 as bit patterns,
 * row-major contiguous arrays, asynchronous on `stream`, argument errors on
 * the host before any launch) with one difference: the WORKSPACE OF THESE
 * CALLS is plain scratch of at least sqllm_moe_workspace_bytes() bytes,
 * 256-byte aligned.  It need not be zero before a call, holds nothing
 * between calls and is left with any contents, so it must not be given to
 * the calls of sqllm.h, which need theirs zeroed.  Calls that may run at
 * the same time need separate workspaces.
 */
#ifndef SQLLM_MOE_H
#define SQLLM_MOE_H

#include "sqllm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SQLLM_MOE_MAX_EXPERTS 512
#define SQLLM_MOE_MAX_TOPK 8

#define SQLLM_MOE_SIGMOID 1  /* scores are sigmoids of the sums, not their softmax */
#define SQLLM_MOE_KEEP_SUM 2 /* the weights are not divided by their sum */

/* One projection of every expert. */
typedef struct {
    const void *packed;      /* [experts] packed matrices of sqllm_packed_bytes() each, 16-byte aligned */
    const uint16_t *lut;     /* fp16 [experts][rows][2^bits], 16-byte aligned */
    const int32_t *row_ptr;  /* int32 [experts * rows + 1]: one CSR over the experts' rows in order */
    const uint16_t *col_idx; /* uint16 [nnz], < cols in the rows' entries */
    const uint16_t *val;     /* fp16 [nnz] */
    int64_t nnz;             /* 0: no outliers (row_ptr, col_idx and val may be NULL); at least row_ptr's last
                              * entry, what the arrays hold behind it is of no row */
} sqllm_experts;

/* Scratch bytes that every call below needs at most for these sizes; 0 if
 * they are out of range.  sqllm_moe_route alone takes inter = 256. */
size_t sqllm_moe_workspace_bytes(int batch, int experts, int topk, int64_t hidden, int64_t inter);

/*
 * sqllm_moe_route -- choose each token's experts and their weights.
 *   x: fp16 [batch][hidden], router: fp16 [experts][hidden], both 16-byte
 *   aligned; bias: fp32 [experts], added to the scores for the choice only
 *   (NULL: none); flags: SQLLM_MOE_SIGMOID | SQLLM_MOE_KEEP_SUM (others are
 *   SQLLM_ERR_SHAPE); ids: int32, weights: fp32, both [batch][topk].
 *   A token's ids are distinct.  A score that is not a number ranks below
 *   every other, those among themselves by the lowest expert.
 */
sqllm_status sqllm_moe_route(const uint16_t *x, const uint16_t *router, const float *bias, int batch, int experts,
                             int64_t hidden, int topk, int flags, float scale, int32_t *ids, float *weights,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * sqllm_moe_experts -- y from given choices.
 *   ids: int32, weights: fp32, both [batch][topk].  An id outside
 *   [0, experts) takes no part, whatever its weight; a token with none left
 *   gets zeros (its x is not read); an id that comes twice counts with the
 *   sum of its weights.  y: fp16 [batch][hidden], 4-byte aligned; must not
 *   overlap an input.
 */
sqllm_status sqllm_moe_experts(const uint16_t *x, const int32_t *ids, const float *weights, const sqllm_experts *gate,
                               const sqllm_experts *up, const sqllm_experts *down, int bits, int batch, int experts,
                               int topk, int64_t hidden, int64_t inter, uint16_t *y, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/*
 * sqllm_moe_layer -- sqllm_moe_route, then sqllm_moe_experts with its
 * choices, which are returned too.  The same bits as the two calls.
 */
sqllm_status sqllm_moe_layer(const uint16_t *x, const uint16_t *router, const float *bias, int flags, float scale,
                             const sqllm_experts *gate, const sqllm_experts *up, const sqllm_experts *down, int bits,
                             int batch, int experts, int topk, int64_t hidden, int64_t inter, int32_t *ids,
                             float *weights, uint16_t *y, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SQLLM_MOE_H */
