/*
 * sgemm_f32_layer.h -- a whole layer of experts for a few tokens, on one MI355X (gfx950).
 *
 * Token t goes through the experts e = ids[t][j] of its `top` choices, each with two or three
 * matrices of one shape:
 *     h[t][j] = act(x[t] * G_e) . (x[t] * U_e)   (element by element), or, without G,
 *               act(x[t] * U_e),
 *     y[t]    = sum over j of weights[t][j] * (h[t][j] * D_e),
 * U and G being width x hidden and D hidden x width.  A choice outside [0, experts) adds
 * nothing; a token without any gets zeros.  That is what sgemm_f32_route_sort(),
 * _gather(), the products by expert and _combine() of sgemm_f32_experts.h compute
 * together, in two kernels in place of six or more (a third sorts more than 64 choices, and
 * one adds the parts of y where few columns leave few work-groups).  Any number of tokens
 * is taken, 64 at a time, but with more than a few for each expert the parts are faster:
 * there the matrices are no longer what has to be read.
 *
 * The matrices are fp32, in 4 bits (sgemm_f32_w4.h) or in 8 bits (sgemm_f32_f8.h: codes
 * times scales; the rows are not put into 8 bits here), G and U in the same form.
 *
 * Ownership, asynchrony and errors are those of sgemm_f32.h (bad arguments are
 * hipErrorInvalidValue with nothing enqueued, among them a size, or tokens*top, above
 * 2^31 - 65537, top above 32 and more blocks than one launch can hold; nothing is
 * allocated and no pointer kept; calls can be captured into a HIP graph).
 *
 * Arithmetic is fp32: x and h enter the products without rounding (with weights in 4 or 8
 * bits but for bits below 2^-133, which are dropped), sums and activations are fp32.
 * Results are bitwise reproducible for fixed arguments.  A NaN or infinity in a token's x or
 * weights makes elements of its row of y NaN or infinite; other rows are not affected.
 *
 * Large values.  With weights in 4 bits what sgemm_f32_w4.h says of them holds for x and h
 * (up to 1.7e35 for groups of 128 and more).  With weights in 8 bits the power of two of a
 * scale enters before the sum over its block, so nothing overflows as long as the sums of
 * the terms have room, and a block with a scale of zero adds nothing; a code times that
 * power of two counts as infinite from 2^128 on and loses its bits below 2^-133.
 */
#ifndef SGEMM_F32_LAYER_H
#define SGEMM_F32_LAYER_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations: z / (1 + exp(-z)); z * (1 + erf(z / sqrt 2)) / 2; max(z, 0). */
#define SGEMM_F32_LAYER_SILU 0
#define SGEMM_F32_LAYER_GELU 1
#define SGEMM_F32_LAYER_RELU 2

/* Forms of matrices. */
#define SGEMM_F32_LAYER_F32 0
#define SGEMM_F32_LAYER_W4 1
#define SGEMM_F32_LAYER_F8 2

/* One stack of `experts` matrices K x N (of the layer's shapes; the struct is read by the
 * call and not kept). */
typedef struct sgemm_f32_layer_matrices {
    int kind;          /* SGEMM_F32_LAYER_* form */
    const void *data;  /* fp32 matrices, or the array that was packed */
    int ld;            /* F32: row stride >= max(1, N), or >= max(1, K) with trans */
    long long stride;  /* F32: elements between matrices, >= 0 */
    int trans;         /* F32: SGEMM_F32_OP_T where the matrices are given as N x K */
    int group;         /* W4: as it was packed with */
    int scale_type;    /* W4: likewise */
    int zeros;         /* W4: likewise */
} sgemm_f32_layer_matrices;

/*
 * ids and weights are tokens x top (row strides ldids, ldw >= max(1, top)), x and y
 * tokens x width (ldx, ldy >= max(1, width)); y is written only.  gate is NULL for a
 * layer without G.  workspace: sgemm_f32_layer_workspace_size() bytes (may be 0), 16-byte
 * aligned; calls that may run at the same time need one each.  y and workspace overlap no
 * other argument.
 */
size_t sgemm_f32_layer_workspace_size(int tokens, int top, int experts, int width, int hidden);
hipError_t sgemm_f32_layer(int tokens, int top, int experts, int width, int hidden, int act,
                           const int *ids, int ldids, const float *weights, int ldw,
                           const float *x, int ldx,
                           const sgemm_f32_layer_matrices *gate,
                           const sgemm_f32_layer_matrices *up,
                           const sgemm_f32_layer_matrices *down,
                           float *y, int ldy,
                           void *workspace, size_t workspace_bytes,
                           hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_LAYER_H */
