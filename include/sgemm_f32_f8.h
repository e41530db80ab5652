/*
 * sgemm_f32_f8.h -- matrix products in 8-bit floating point with a scale for each
 * block of 128, on one MI355X (gfx950).
 *
 * Both operands are 8-bit floating-point codes: e4m3 (largest number 448) or e5m2
 * (57344).  Weights W (K x N) have one scale for each block of 128 k by 128 columns,
 *     W[k][n] = sw[k / 128][n / 128] * qw[k][n]        (qw: e4m3),
 * and rows A (rows x K) are put into 8 bits with one scale for each row and block of
 * 128 k,
 *     A8[i][k] = sa[i][k / 128] * qa[i][k],
 *     sa = the smallest power of two with max|A| over the block <= 448 * sa (e4m3) or
 *          57344 * sa (e5m2), at least 2^-124 (2^-117); 1 where all of them are zero,
 *     qa = A / sa rounded to the nearest code, ties to even (the division is exact).
 * The product is
 *     C[i][n] = sum over k of A8[i][k] * W[k][n].
 * The gradient of the weights is a product of the same kind whose sums run over the
 * rows: both operands are put into 8 bits along their columns, in blocks of 128 rows
 * of an expert (sgemm_f32_f8_ta).  A product with few rows is bound by the bytes of W
 * (the intensity formula of page "CUDA算子优化(4)：矩阵乘法", section "计算强度"), and
 * W has a quarter of the bytes of an fp32 B.
 *
 * Ownership, asynchrony and errors are those of sgemm_f32.h (bad arguments are
 * hipErrorInvalidValue with nothing enqueued, among them a size above 2^31 - 65537
 * and more blocks than one launch can hold; nothing is allocated and no pointer
 * kept; calls can be captured into a HIP graph).
 *
 * Arithmetic.  Products of codes and powers of two are exact and are added in fp32, for
 * results of either type; a bf16 result is rounded once from that (to nearest, ties to
 * even).  Of an fp32 scale of the weights what is not a power of two multiplies a block's
 * sum before it is added.  Results are bitwise reproducible for fixed arguments.
 *
 * Values.  A NaN or infinite A[i][k] gets the code NaN and makes row i of the result
 * NaN (in sgemm_f32_f8_ta row or column i of its expert's matrix); other rows are not
 * affected.  A NaN code or scale of W makes its columns NaN, an infinite scale
 * NaN or infinite; a block with a scale of zero adds nothing, however large the rows.
 * Values of A that round to 2^128 in 8 bits (1.9375 * 2^127, 3.296e38, and more) count as
 * infinite: their rows of the result become infinite or NaN.  Values of A below
 * 2^-134 become zero, and below 2^-130 (e4m3) or 2^-131 (e5m2) they have fewer bits
 * than codes have.  A code of W times the power of two in its scale counts as infinite from
 * 2^128 on and loses its bits below 2^-133.  Beyond that a block's sum is formed with the
 * powers of two of both scales and then multiplied by what is left of W's, 1 to 2, so
 * nothing overflows as long as the sums of the terms have room.
 */
#ifndef SGEMM_F32_F8_H
#define SGEMM_F32_F8_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of codes. */
#define SGEMM_F32_F8_E4M3 0
#define SGEMM_F32_F8_E5M2 1

/* Type of the rows that are given, and of results (F32 or BF16). */
#define SGEMM_F32_F8_IN_F32 0
#define SGEMM_F32_F8_IN_BF16 1
#define SGEMM_F32_F8_IN_ROWS 2 /* an array that sgemm_f32_f8_rows() has written */

/* Type of the scales of weights: fp32 numbers, or powers of two (a byte b is
 * 2^(b - 127), 255 is NaN). */
#define SGEMM_F32_F8_SCALE_F32 0
#define SGEMM_F32_F8_SCALE_E8M0 1

/*
 * Weights are laid out once, for `experts` >= 1 matrices of one shape (1 for a
 * single matrix), into one device array that the products read.
 *
 * sgemm_f32_f8_packed_size()  bytes of that array (0 for invalid arguments).
 * sgemm_f32_f8_pack()         from codes and scales:
 *     codes   matrix e at codes + e*stride, K x N with row stride ld >= max(1, N)
 *             or, with trans = SGEMM_F32_OP_T, N x K with ld >= max(1, K);
 *     scales  experts x ceil(K/128) x ceil(N/128) values of scale_type, or
 *             experts x ceil(N/128) x ceil(K/128) with trans.
 * sgemm_f32_f8_quantize()     from fp32 matrices (laid out as codes above), with the
 *     formula of the rows over each 128 x 128: codes e4m3, scales powers of two (a
 *     product takes the array as SCALE_E8M0).  `packed` gets the matrices,
 *     `packed_t` their transposes (N x K, for products with the gradient; of
 *     sgemm_f32_f8_packed_size(experts, K, N) bytes); either may be NULL.
 * sgemm_f32_f8_unpack()       the fp32 matrices that the packed array stands for,
 *     each code times its scale rounded to fp32.
 * packed arrays are 16-byte aligned, of at least that size (the bytes given are
 * checked) and overlap no other argument.
 */
size_t sgemm_f32_f8_packed_size(int experts, int N, int K);
hipError_t sgemm_f32_f8_pack(int experts, int N, int K, int trans,
                             const unsigned char *codes, int ld, long long stride,
                             const void *scales, int scale_type,
                             void *packed, size_t packed_bytes,
                             hipStream_t stream);
hipError_t sgemm_f32_f8_quantize(int experts, int N, int K, int trans,
                                 const float *B, int ldb, long long strideb,
                                 void *packed, size_t packed_bytes,
                                 void *packed_t, size_t packed_t_bytes,
                                 hipStream_t stream);
hipError_t sgemm_f32_f8_unpack(int experts, int N, int K,
                               const void *packed, size_t packed_bytes,
                               float *B, int ldb, long long strideb,
                               hipStream_t stream);

/*
 * Rows in 8 bits, for several products with the same rows: q gets
 * sgemm_f32_f8_rows_size() bytes (0 for invalid arguments), 16-byte aligned.
 * A is rows x K numbers of in_type (F32 or BF16), lda >= max(1, K).
 */
size_t sgemm_f32_f8_rows_size(int rows, int K);
hipError_t sgemm_f32_f8_rows(int rows, int K, const void *A, int lda, int in_type, int code_type,
                             void *q, size_t q_bytes, hipStream_t stream);

/*
 * C = A8 * W for one matrix (offsets == NULL, experts == 1), or by expert: C[i] =
 * A8[i] * W_e for every row i of expert e (offsets[e] <= i < offsets[e+1]; experts + 1
 * values on the device, as sgemm_f32_route_sort() of sgemm_f32_experts.h writes them,
 * clamped as described there).  Rows of no expert are left as they are.
 *   A      rows x K numbers of in_type with row stride lda >= max(1, K), put into
 *          codes of code_type; or with SGEMM_F32_F8_IN_ROWS the array of
 *          sgemm_f32_f8_rows(rows, K, ..., code_type), 16-byte aligned (lda is not read);
 *   C      rows x N (ldc >= max(1, N)) of out_type F32 or BF16, written only.
 *          K == 0 writes zeros;
 *   workspace  of sgemm_f32_f8_workspace_size() bytes (which may be 0, and is for
 *          SGEMM_F32_F8_IN_ROWS), 16-byte aligned; calls that may run at the same time
 *          need one each.
 */
size_t sgemm_f32_f8_workspace_size(int rows, int N, int K, int experts, int by_expert);
hipError_t sgemm_f32_f8(int rows, int N, int K, int experts, const int *offsets,
                        const void *A, int lda, int in_type, int code_type,
                        const void *packed, int scale_type,
                        void *C, int ldc, int out_type,
                        void *workspace, size_t workspace_bytes,
                        hipStream_t stream);

/*
 * C_e = alpha * A8_e^T * D8_e + beta * C_e over the rows of each expert (offsets == NULL,
 * experts == 1: over all rows): the gradient of the weights, for D = the gradient of the
 * result.  A is rows x M and D rows x N numbers of their in_types (F32 or BF16), put into
 * codes of their code_types along their columns, with one scale for each column and
 * block of 128 of an expert's rows, the first block beginning with its first row.  Matrix
 * e of C is M x N fp32 at C + e*stridec; an expert without rows gets beta * C_e.
 * beta == 0 means C is not read.  The workspace is as above.
 */
size_t sgemm_f32_f8_ta_workspace_size(int rows, int M, int N, int experts);
hipError_t sgemm_f32_f8_ta(int rows, int M, int N, int experts, const int *offsets, float alpha,
                           const void *A, int lda, int a_in_type, int a_code_type,
                           const void *D, int ldd, int d_in_type, int d_code_type,
                           float beta, float *C, int ldc, long long stridec,
                           void *workspace, size_t workspace_bytes,
                           hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_F8_H */
