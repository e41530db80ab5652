/*
 * sgemm_f32_experts.h -- products of several matrices in one call, and the
 * ordering of rows around them, on one MI355X (gfx950).
 *
 * A layer of experts sends every token (a row of activations) to `top` of
 * `experts` weight matrices, and adds the results with a weight for each.  The
 * entry points here are its parts:
 *   sgemm_f32_route_sort()          which row goes where: the (token, choice)
 *                                   pairs in the order of their experts;
 *   sgemm_f32_route_gather()        the tokens' rows in that order;
 *   sgemm_f32_grouped()             the products, one launch for all experts;
 *   sgemm_f32_route_combine()       each token's rows back, weighted and added;
 *   sgemm_f32_route_combine_grad()  the gradient of that with respect to the
 *                                   rows and the weights;
 *   sgemm_f32_grouped_ta()          the gradient of the products with respect to
 *                                   the experts' matrices.
 * The gradient of sgemm_f32_route_gather() is sgemm_f32_route_combine() without
 * weights, and that of sgemm_f32_grouped() with respect to its rows is
 * sgemm_f32_grouped() with the matrices transposed.
 *
 * Ownership, asynchrony and errors are those of sgemm_f32.h: the caller owns
 * every buffer, the library allocates nothing and keeps no pointer, each call
 * validates its arguments on the host, enqueues its kernels on `stream` and
 * returns without waiting, and a bad argument is hipErrorInvalidValue with
 * nothing enqueued: a negative size, a leading dimension below the row length, a
 * NULL buffer that would be used, a written array overlapping any other, a size
 * (or tokens*top) above 2^31 - 65537, more blocks than one launch can hold.  Sizes
 * of zero enqueue nothing (unless an output still has to be written).  Calls can
 * be captured into a HIP graph.  Results are bitwise reproducible: no result
 * depends on the order in which work-groups run.
 *
 * What the device arrays hold is not known to the host and is checked by the
 * kernels: an expert id outside [0, experts) drops its pair; a place or pair
 * number outside its array is treated as dropped; offsets are clamped to
 * 0 <= offsets[e] <= offsets[e+1] <= rows, so no content of these arrays makes a
 * kernel leave the arrays it was given.  (Offsets whose clamped ranges overlap, or
 * a position that several pairs have, which sgemm_f32_route_sort() never writes,
 * make several experts or pairs write the same rows, with an unspecified result
 * there.)
 *
 * Arithmetic is IEEE fp32 with fused multiply-adds, as in sgemm_f32.h.
 */
#ifndef SGEMM_F32_EXPERTS_H
#define SGEMM_F32_EXPERTS_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The order of rows by expert.  Pair f = t*top + j is token t's choice j, for
 * expert ids[t*ldids + j].
 *   offsets   experts + 1 values: offsets[e] pairs have an expert below e, so
 *             expert e's rows are offsets[e] .. offsets[e+1]-1, and
 *             offsets[experts] pairs are kept.
 *   order     tokens*top values: the pair at each place, by expert and, within
 *             an expert, by pair number; -1 from place offsets[experts] on.
 *   position  tokens*top values: each pair's place in `order`; -1 if dropped.
 * ldids >= max(1, top).  The workspace (device
 * memory, 16-byte aligned, contents irrelevant before and after) must hold
 * sgemm_f32_route_workspace_size() bytes, which may be 0 (then it may be NULL);
 * calls that overlap in time must not share it.  The size is 0 for invalid
 * arguments too.
 * The pairs are walked twice for up to 895 experts, and twice for each digit of the
 * experts' numbers beyond (two digits up to 802815 experts, at most four), but for
 * a few thousand pairs of a few thousand experts, which one launch sorts.
 */
size_t sgemm_f32_route_workspace_size(int tokens, int top, int experts);
hipError_t sgemm_f32_route_sort(int tokens, int top, int experts,
                                const int *ids, int ldids,
                                int *offsets, int *order, int *position,
                                void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/*
 * rows[position[f]] = x[f / top] for every pair f with a place; other rows are
 * left as they are.  x is tokens x width (row stride ldx >= max(1, width)), rows is
 * tokens*top x width (ldrows >= max(1, width)).
 */
hipError_t sgemm_f32_route_gather(int tokens, int top, int width, const int *position,
                                  const float *x, int ldx,
                                  float *rows, int ldrows,
                                  hipStream_t stream);

/*
 * out[t] = sum over j = 0 .. top-1 of weights[t*ldw + j] * rows[position[t*top + j]],
 * added in the order of j; a pair with position -1 adds nothing, and a token
 * whose pairs are all dropped gets zeros.  weights == NULL means 1 for every
 * pair (ldw is then not used).  ldw >= max(1, top), ldrows and ldout >=
 * max(1, width).
 */
hipError_t sgemm_f32_route_combine(int tokens, int top, int width, const int *position,
                                   const float *weights, int ldw,
                                   const float *rows, int ldrows,
                                   float *out, int ldout,
                                   hipStream_t stream);

/*
 * The gradient of sgemm_f32_route_combine(), given dout = the gradient of out:
 *   drows[position[f]] = weights[t, j] * dout[t]       (rows of no pair: left as they are)
 *   dweights[t, j]     = sum over columns of dout[t] * rows[position[f]]   (0 if dropped)
 * for f = t*top + j.  Either of drows and dweights may be NULL (not wanted);
 * rows is read only for dweights and may be NULL without it.  weights == NULL
 * means 1 for every pair.  dweights has the row stride ldw, as weights.
 */
hipError_t sgemm_f32_route_combine_grad(int tokens, int top, int width, const int *position,
                                        const float *weights, int ldw,
                                        const float *rows, int ldrows,
                                        const float *dout, int lddout,
                                        float *drows, int lddrows,
                                        float *dweights,
                                        hipStream_t stream);

/*
 * C[i] = alpha * A[i] * op(B_e) + beta * C[i] for every row i of expert e
 * (offsets[e] <= i < offsets[e+1], offsets on the device), one launch for all
 * experts.  A is rows x K (lda >= max(1, K)), C is rows x N (ldc >= max(1, N)).
 * B_e starts at B + e*strideb: K x N with row stride ldb >= max(1, N) for
 * transb = SGEMM_F32_OP_N, N x K with ldb >= max(1, K) for SGEMM_F32_OP_T.  The
 * experts' matrices may be one and the same (strideb == 0) but strideb must not
 * be negative.  Rows of no expert (from offsets[experts] on, or before offsets[0])
 * are left as they are.  beta == 0 means C is not read; alpha == 0 or K == 0
 * means A and B are not read.
 */
hipError_t sgemm_f32_grouped(int transb, int rows, int N, int K, int experts,
                             const int *offsets, float alpha,
                             const float *A, int lda,
                             const float *B, int ldb, long long strideb, float beta,
                             float *C, int ldc,
                             hipStream_t stream);

/*
 * C_e = alpha * A_e^T * D_e + beta * C_e for every expert e, where A_e and D_e
 * are the rows offsets[e] .. offsets[e+1]-1 of A (rows x M, lda >= max(1, M)) and D
 * (rows x N, ldd >= max(1, N)), and C_e is the M x N array at C + e*stridec
 * (ldc >= max(1, N), stridec at least the extent of one C_e).  An expert without
 * rows gets beta * C_e (zeros for beta == 0).
 */
hipError_t sgemm_f32_grouped_ta(int rows, int M, int N, int experts,
                                const int *offsets, float alpha,
                                const float *A, int lda,
                                const float *D, int ldd, float beta,
                                float *C, int ldc, long long stridec,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_EXPERTS_H */
