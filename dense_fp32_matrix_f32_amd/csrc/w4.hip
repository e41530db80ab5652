// w4.hip -- fp32 rows times a matrix of 4-bit weights.
//
//     C[i][n] = sum over groups g of s[g][n] * sum over k in g of A[i][k] * (q[k][n] - z[g][n])
//
// The simplest form: one work-item for each element of C, the k loop in registers.
#include "groups.h"
#include "w4.h"

namespace sgemm {

namespace {

__global__ __launch_bounds__(256) void w4_kernel(W4Layout l, W4Problem p) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    for (int i = blockIdx.y; i < p.rows; i += gridDim.y) {
        int e = 0;
        if (p.offsets) {
            int first, end;
            if (!find_block(p.offsets, p.experts, p.rows, 1, i, &e, &first, &end)) return;
            if (n < l.N) {
                // block i of one row each is row `first`
                const float *a = p.A + (int64_t)first * p.lda;
                float sum = 0.0f;
                const unsigned char *strip = p.packed + e * l.expert_bytes +
                                             (int64_t)(n / kW4Cols) * l.strip_bytes;
                for (int k = 0; k < l.K; ++k) {
                    const unsigned char *rec = strip + (int64_t)(k / kW4Block) * l.record;
                    const int kb = k % kW4Block, c = n % kW4Cols;
                    const unsigned word =
                        *(const unsigned *)(rec + 16 * (c + 16 * (kb % 32 / 8)) + 4 * (kb / 32));
                    const int at = kb / (kW4Block / l.parts) * kW4Cols + c;
                    const float s = w4_scale(rec + kW4Codes + at * l.scale_size, l.scale_type);
                    const int z =
                        l.zeros ? rec[kW4Codes + l.parts * kW4Cols * l.scale_size + at] : 8;
                    sum = fmaf(a[k], s * (float)((int)(word >> w4_shift(kb % 8) & 15) - z), sum);
                }
                p.C[(int64_t)first * p.ldc + n] = sum;
            }
            continue;
        }
        if (n >= l.N) continue;
        const float *a = p.A + (int64_t)i * p.lda;
        float sum = 0.0f;
        const unsigned char *strip = p.packed + (int64_t)(n / kW4Cols) * l.strip_bytes;
        for (int k = 0; k < l.K; ++k) {
            const unsigned char *rec = strip + (int64_t)(k / kW4Block) * l.record;
            const int kb = k % kW4Block, c = n % kW4Cols;
            const unsigned word =
                *(const unsigned *)(rec + 16 * (c + 16 * (kb % 32 / 8)) + 4 * (kb / 32));
            const int at = kb / (kW4Block / l.parts) * kW4Cols + c;
            const float s = w4_scale(rec + kW4Codes + at * l.scale_size, l.scale_type);
            const int z = l.zeros ? rec[kW4Codes + l.parts * kW4Cols * l.scale_size + at] : 8;
            sum = fmaf(a[k], s * (float)((int)(word >> w4_shift(kb % 8) & 15) - z), sum);
        }
        p.C[(int64_t)i * p.ldc + n] = sum;
    }
}

}  // namespace

hipError_t launch_w4(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    const dim3 grid((unsigned)((l.N + 255ll) / 256), (unsigned)(p.rows < 65535 ? p.rows : 65535));
    return launch(w4_kernel, grid, dim3(256), 0, s, l, p);
}

}  // namespace sgemm
