// w4_pack.hip -- 4-bit weights into the layout of w4.h and back.  These run once for a
// set of weights and are simple rather than fast; none reaches the rate of a copy (5.0
// TB/s).  With f16 scales, in us, the bytes counted once:
//   matrices, group             pack             quantize         unpack
//    1 of 4096 x 4096,   32     10 (1.8 TB/s)      41 (1.9)        70 (1.1)
//    1 of 4096 x 4096,  128     10 (1.8)           91 (0.8)        70 (1.1)
//    1 of 4096 x 4096, 4096     10 (1.7)         2480 (0.03)       72 (1.1)
//   64 of 2048 x 2048,  128    124 (2.2)          731 (1.7)       890 (1.4)
//    8 of 8192 x 8192,  128    357 (1.6)         1437 (1.7)      1758 (1.4)
#include "w4.h"

namespace sgemm {

namespace {

// One wave for each record, lane l as in w4.h.  Codes past K are 8 and the scales
// of columns past N are 0; neither meets a stored result.
__global__ __launch_bounds__(256) void pack_kernel(W4Layout l, int64_t records,
                                                   const unsigned char *__restrict__ codes,
                                                   const unsigned char *__restrict__ scales,
                                                   const unsigned char *__restrict__ zeros,
                                                   unsigned char *__restrict__ packed) {
    const int lane = threadIdx.x & 63;
    const int groups = (int)(((int64_t)l.K + l.group - 1) / l.group);
    const int64_t pairs = ((int64_t)l.K + 1) / 2;
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < records;
         r += (int64_t)gridDim.x * 4) {
        const int b = (int)(r % l.blocks);
        const int64_t es = r / l.blocks;
        const int strip = (int)(es % l.strips);
        const int64_t e = es / l.strips;
        const int n = strip * kW4Cols + lane % 16, q = lane / 16;
        unsigned char *rec = packed + r * l.record;
        unsigned word[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            word[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int64_t k = (int64_t)b * kW4Block + 32 * j + w4_k(q, i);
                unsigned byte = 0x88;
                if (n < l.N && k < l.K) {
                    byte = codes[(e * pairs + k / 2) * l.N + n];
                    if (k + 1 >= l.K) byte = (byte & 15) | 0x80;
                }
                word[j] |= (byte & 15) << w4_shift(i);
                word[j] |= (byte >> 4) << w4_shift(i + 1);
            }
        }
        *(uint4 *)(rec + 16 * lane) = uint4{word[0], word[1], word[2], word[3]};
        if (q < l.parts) {
            const int64_t g = ((int64_t)b * kW4Block + (int64_t)q * (kW4Block / l.parts)) / l.group;
            const bool in = n < l.N && g < groups;
            const int64_t at = in ? (e * groups + g) * l.N + n : 0;
            const int place = lane % 16 * l.parts + q;
            unsigned char *s = rec + kW4Codes + place * l.scale_size;
            if (l.scale_size == 4) {
                *(unsigned *)s = in ? ((const unsigned *)scales)[at] : 0;
            } else {
                *(unsigned short *)s = in ? ((const unsigned short *)scales)[at] : 0;
            }
            if (l.zeros)
                rec[kW4Codes + l.parts * kW4Cols * l.scale_size + place] =
                    in ? zeros[at] : 0;
        }
    }
}

// One work-item for each group of a column: its extremes, then its codes, so B is read
// twice, and groups of many k leave few work-items, each waiting for its loads.
__global__ __launch_bounds__(256) void quantize_kernel(W4Layout l, int64_t items, int groups,
                                                       const float *__restrict__ B, int64_t ldb,
                                                       int64_t strideb,
                                                       unsigned char *__restrict__ packed) {
    const int cols = l.strips * kW4Cols;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items;
         it += (int64_t)gridDim.x * 256) {
        const int n = (int)(it % cols);
        const int64_t eg = it / cols;
        const int g = (int)(eg % groups);
        const int64_t e = eg / groups;
        const int64_t k0 = (int64_t)g * l.group;
        // groups past K fill the last block's places
        const int64_t k1 = min(k0 + l.group, (int64_t)l.blocks * kW4Block);
        const int64_t kend = n < l.N ? min(k1, (int64_t)l.K) : k0;
        const float *col = B + e * strideb + n;
        float lo = 0.0f, hi = 0.0f;
        for (int64_t k = k0; k < kend; ++k) {
            const float x = col[k * ldb];
            lo = fminf(lo, x);
            hi = fmaxf(hi, x);
        }
        const float wide = l.zeros ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
        float s = 0.0f;
        int z = 8;
        unsigned char *strip = packed + e * l.expert_bytes + (int64_t)(n / kW4Cols) * l.strip_bytes;
        for (int64_t k = k0; k < k1; k += kW4Block) {
            const int64_t b = k / kW4Block;
            const int part = l.parts > 1 ? (int)(k % kW4Block) / l.group : 0;
            unsigned char *rec = strip + b * l.record;
            const int at = n % kW4Cols * l.parts + part;
            s = w4_store_scale(rec + kW4Codes + at * l.scale_size, wide, l.scale_type);
            if (l.zeros) {
                z = s > 0.0f ? (int)fminf(rintf(-lo / s), 15.0f) : 8;
                rec[kW4Codes + l.parts * kW4Cols * l.scale_size + at] = (unsigned char)z;
            }
            const int len = min(l.group, kW4Block);
            for (int w = 0; w < len / 8; ++w) {
                const int from = w / 4 * 32;  // this word's 32 k, from the part's first on
                unsigned word = 0;
                for (int i = 0; i < 8; ++i) {
                    const int64_t ki = k + from + w4_k(w % 4, i);
                    int q = z;
                    if (ki < kend && s > 0.0f)
                        q = (int)fminf(fmaxf(rintf(col[ki * ldb] / s) + z, 0.0f), 15.0f);
                    word |= (unsigned)q << w4_shift(i);
                }
                *(unsigned *)(rec + 16 * (n % kW4Cols + 16 * (w % 4)) +
                              4 * ((part * len + from) / 32)) = word;
            }
        }
    }
}

// One work-item for each element.
__global__ __launch_bounds__(256) void unpack_kernel(W4Layout l, int64_t items,
                                                     const unsigned char *__restrict__ packed,
                                                     float *__restrict__ B, int64_t ldb,
                                                     int64_t strideb) {
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items;
         it += (int64_t)gridDim.x * 256) {
        const int n = (int)(it % l.N);
        const int64_t ek = it / l.N;
        const int k = (int)(ek % l.K);
        const int64_t e = ek / l.K;
        const unsigned char *rec = packed + e * l.expert_bytes +
                                   (int64_t)(n / kW4Cols) * l.strip_bytes +
                                   (int64_t)(k / kW4Block) * l.record;
        const int kb = k % kW4Block, c = n % kW4Cols;
        const unsigned word =
            *(const unsigned *)(rec + 16 * (c + 16 * w4_part(kb % 32)) + 4 * (kb / 32));
        const int at = c * l.parts + kb / (kW4Block / l.parts);
        const float s = w4_scale(rec + kW4Codes + at * l.scale_size, l.scale_type);
        const int z = l.zeros ? rec[kW4Codes + l.parts * kW4Cols * l.scale_size + at] : 8;
        const int q = (word >> w4_shift(w4_index(kb % 32))) & 15;
        B[e * strideb + k * ldb + n] = s * (float)(q - z);
    }
}

unsigned grid_for(int64_t groups) { return (unsigned)(groups < 65536 ? groups : 65536); }

}  // namespace

hipError_t launch_w4_pack(const W4Layout &l, int experts, const unsigned char *codes,
                          const unsigned char *scales, const unsigned char *zeros,
                          unsigned char *packed, hipStream_t s) {
    const int64_t records = (int64_t)experts * l.strips * l.blocks;
    return launch(pack_kernel, dim3(grid_for((records + 3) / 4)), dim3(256), 0, s, l, records,
                  codes, scales, zeros, packed);
}

hipError_t launch_w4_quantize(const W4Layout &l, int experts, const float *B, int64_t ldb,
                              int64_t strideb, unsigned char *packed, hipStream_t s) {
    const int64_t whole = (int64_t)l.blocks * kW4Block;
    const int groups = (int)((whole + l.group - 1) / l.group);
    const int64_t items = (int64_t)experts * groups * l.strips * kW4Cols;
    return launch(quantize_kernel, dim3(grid_for((items + 255) / 256)), dim3(256), 0, s, l, items,
                  groups, B, ldb, strideb, packed);
}

hipError_t launch_w4_unpack(const W4Layout &l, int experts, const unsigned char *packed, float *B,
                            int64_t ldb, int64_t strideb, hipStream_t s) {
    const int64_t items = (int64_t)experts * l.K * l.N;
    return launch(unpack_kernel, dim3(grid_for((items + 255) / 256)), dim3(256), 0, s, l, items,
                  packed, B, ldb, strideb);
}

}  // namespace sgemm
