/*
 * sgemm_f32_w4.h -- products of fp32 rows with matrices kept in 4 bits, on one
 * MI355X (gfx950).
 *
 * A K x N matrix W is held as 4-bit codes q with a scale (and, if wanted, a zero
 * point) for each `group` consecutive values of a column:
 *     W[k][n] = s[k / group][n] * (q[k][n] - z[k / group][n]),
 * q in 0 .. 15, z a byte (8 where there are no zero points).  The product is
 *     C[i][n] = sum over k of A[i][k] * W[k][n],
 * the definition of sgemm_f32.h with B = W.  A product with few rows is bound by
 * the bytes of B (the intensity formula of page "CUDA算子优化(4)：矩阵乘法",
 * section "计算强度"), and W has about an eighth of the bytes of an fp32 B.
 *
 * Ownership, asynchrony and errors are those of sgemm_f32.h (bad arguments are
 * hipErrorInvalidValue with nothing enqueued, among them a size above 2^31 - 65537
 * and more blocks than one launch can hold; nothing is allocated and no pointer
 * kept; calls can be captured into a HIP graph).
 *
 * Arithmetic.  Sums are fp32: for each group the sum of A[i][k] * q less z times the
 * sum of A[i][k], times s.  Rounding errors are thus relative to |A[i][k]| * s *
 * (q + z) rather than to |q - z|, and results are as accurate as fp32 products of
 * such terms.  The inputs enter without rounding, but bits of A[i][k] below 2^-133
 * (1e-40) are dropped, so values from 2^-110 (8e-34) on lose nothing.  Results are
 * bitwise reproducible for fixed arguments.
 *
 * Large values.  The sums over a group, or over 128 of its k at a time, are formed
 * before s meets them.  Nothing overflows as long as the result, and s times such a
 * sum, have room and |A[i][k]| is at most 2.2e37 / min(group, 128): 1.7e35 for groups
 * of 128 and more, 3.4e35 for 64 and 6.8e35 for 32 (1.3e36 / min(group, 128) with zero
 * points above 15).  Beyond that an element can become infinite or NaN.  A NaN or
 * infinite A[i][k] makes all of row i NaN or infinite (NaN also where the definition
 * has an infinity).  Other rows are not affected.
 *
 * Groups.  `group` is 32, 64 or a multiple of 128 (any such value from K on
 * means one group for each column); the last group may be cut short by K.
 */
#ifndef SGEMM_F32_W4_H
#define SGEMM_F32_W4_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the scales. */
#define SGEMM_F32_W4_SCALE_F32 0
#define SGEMM_F32_W4_SCALE_F16 1
#define SGEMM_F32_W4_SCALE_BF16 2

/*
 * Weights are laid out once, for `experts` >= 1 matrices of one shape (1 for a
 * single matrix), into one device array that the products read.
 *
 * sgemm_f32_w4_packed_size()  bytes of that array (0 for invalid arguments).
 *                             zeros != 0: with zero points.
 * sgemm_f32_w4_pack()         from codes, scales and zero points:
 *     codes   experts x ceil(K/2) x N bytes; byte [k/2][n] holds q[k][n] in its
 *             low four bits for even k, in its high four bits for odd k;
 *     scales  experts x ceil(K/group) x N values of scale_type;
 *     zeros   experts x ceil(K/group) x N bytes, or NULL (8 everywhere).
 * sgemm_f32_w4_quantize()     from fp32 matrices: matrix e is K x N at
 *     B + e*strideb with row stride ldb >= max(1, N).  For each group:
 *       without zero points  s = max|B| / 7 rounded to scale_type,
 *                            q = min(max(rint(B / s) + 8, 0), 15);
 *       with zero points     lo = min(0, min B), hi = max(0, max B),
 *                            s = (hi - lo) / 15 rounded to scale_type,
 *                            z = min(rint(-lo / s), 15),
 *                            q = min(max(rint(B / s) + z, 0), 15);
 *     computed in fp32; where s is 0, q = z (= 8 without zero points).  B has to
 *     be finite, and s within the range of scale_type.
 * sgemm_f32_w4_unpack()       the fp32 matrices that the packed array stands for
 *     (for products with sgemm_f32(), or inspection).
 * packed is 16-byte aligned, of at least sgemm_f32_w4_packed_size() bytes
 * (packed_bytes is checked) and overlaps no other argument.
 */
size_t sgemm_f32_w4_packed_size(int experts, int N, int K, int group, int scale_type, int zeros);
hipError_t sgemm_f32_w4_pack(int experts, int N, int K, int group,
                             const unsigned char *codes, const void *scales, int scale_type,
                             const unsigned char *zeros,
                             void *packed, size_t packed_bytes,
                             hipStream_t stream);
hipError_t sgemm_f32_w4_quantize(int experts, int N, int K, int group,
                                 const float *B, int ldb, long long strideb,
                                 int scale_type, int zeros,
                                 void *packed, size_t packed_bytes,
                                 hipStream_t stream);
hipError_t sgemm_f32_w4_unpack(int experts, int N, int K, int group, int scale_type, int zeros,
                               const void *packed, size_t packed_bytes,
                               float *B, int ldb, long long strideb,
                               hipStream_t stream);

/*
 * C = A * W for one matrix.  A is M x K (lda >= max(1, K)), C is M x N (ldc >=
 * max(1, N)), written only; group, scale_type and zeros are those the array was
 * packed with.  K == 0 writes zeros.
 */
hipError_t sgemm_f32_w4(int M, int N, int K,
                        const float *A, int lda,
                        const void *packed, int group, int scale_type, int zeros,
                        float *C, int ldc,
                        hipStream_t stream);

/*
 * C[i] = A[i] * W_e for every row i of expert e (offsets[e] <= i <
 * offsets[e+1]; experts + 1 values on the device, as sgemm_f32_route_sort()
 * of sgemm_f32_experts.h writes them, clamped as described there).  Rows of no
 * expert are left as they are.
 */
hipError_t sgemm_f32_w4_experts(int rows, int N, int K, int experts, const int *offsets,
                                const float *A, int lda,
                                const void *packed, int group, int scale_type, int zeros,
                                float *C, int ldc,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_W4_H */
