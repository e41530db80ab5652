// w4.h -- how 4-bit weights are laid out on the device, shared by the packing
// kernels and the product.
//
// A matrix is cut into strips of 16 columns and each strip into blocks of 128 k.
// A block is one record: 1024 bytes of codes, then its scales, then its zero
// points (if any).  The 16 bytes at 16*lane belong to column lane % 16; word j of
// them holds the codes of k = 32*j + 4*q + 0 .. 3 and 32*j + 16 + 4*q + 0 .. 3, q =
// lane / 16, so one 16-byte load a lane fetches a block and its word j is the lane's
// operand of the j-th 16x16x32 matrix instruction (which adds over k in any order that
// both operands share; in this one the lanes of a row of A load 64 bytes side by
// side).  Within a word, codes 0 .. 3 are the low
// halves of bytes 0 .. 3 and codes 4 .. 7 their high halves: two masks give
// eight bytes, each the code itself.  Scales and zero points are [column][part]
// with one part for each min(group, 128) values of k, so a lane fetches those of
// its column with one load each; a group longer than a block has its scale in
// each of its blocks (2 to 5 bytes for 64 of codes), so a strip is read as one
// run of memory with nothing on the side.
#pragma once

#include "internal.h"

namespace sgemm {

constexpr int kW4Cols = 16;        // columns of a strip
constexpr int kW4Block = 128;      // k of a block
constexpr int kW4Codes = 1024;     // bytes of a block's codes

enum { W4_F32 = 0, W4_F16 = 1, W4_BF16 = 2 };

struct W4Layout {
    int N, K, group, scale_type, zeros;
    int parts;          // scales of a column in a block: 128 / min(group, 128)
    int strips, blocks; // ceil(N / 16), ceil(K / 128)
    int scale_size;     // bytes of a scale
    int record;         // bytes of a block
    int64_t strip_bytes, expert_bytes;
};

inline W4Layout w4_layout(int N, int K, int group, int scale_type, int zeros) {
    W4Layout l;
    l.N = N;
    l.K = K;
    l.group = group;
    l.scale_type = scale_type;
    l.zeros = zeros != 0;
    l.parts = group < kW4Block ? kW4Block / group : 1;
    l.strips = (int)(((int64_t)N + kW4Cols - 1) / kW4Cols);
    l.blocks = (int)(((int64_t)K + kW4Block - 1) / kW4Block);
    l.scale_size = scale_type == W4_F32 ? 4 : 2;
    l.record = kW4Codes + l.parts * kW4Cols * (l.scale_size + l.zeros);
    l.strip_bytes = (int64_t)l.blocks * l.record;
    l.expert_bytes = l.strips * l.strip_bytes;
    return l;
}

__device__ __forceinline__ float w4_scale(const unsigned char *p, int scale_type) {
    if (scale_type == W4_F32) return *(const float *)p;
    const unsigned short bits = *(const unsigned short *)p;
    if (scale_type == W4_F16) return (float)__builtin_bit_cast(_Float16, bits);
    return __builtin_bit_cast(float, (unsigned)bits << 16);
}

// x rounded to scale_type (to nearest, ties to even), stored at p.
__device__ __forceinline__ float w4_store_scale(unsigned char *p, float x, int scale_type) {
    if (scale_type == W4_F32) {
        *(float *)p = x;
    } else if (scale_type == W4_F16) {
        *(_Float16 *)p = (_Float16)x;
    } else {
        *(__bf16 *)p = (__bf16)x;
    }
    return w4_scale(p, scale_type);
}

// k of code i of lane part q within its 32 k, and back.
__host__ __device__ constexpr int w4_k(int q, int i) { return 16 * (i / 4) + 4 * q + i % 4; }
__host__ __device__ constexpr int w4_part(int k) { return k % 16 / 4; }
__host__ __device__ constexpr int w4_index(int k) { return 4 * (k / 16) + k % 4; }

// Place of code i of a word.
__host__ __device__ constexpr int w4_shift(int i) { return i < 4 ? 8 * i : 8 * (i - 4) + 4; }

// A call's product: rows of A, by expert where offsets is not NULL.
struct W4Problem {
    int rows;
    const float *A;
    int64_t lda;
    const unsigned char *packed;
    float *C;
    int64_t ldc;
    int experts;
    const int *offsets;
};

hipError_t launch_w4_pack(const W4Layout &l, int experts, const unsigned char *codes,
                          const unsigned char *scales, const unsigned char *zeros,
                          unsigned char *packed, hipStream_t s);
hipError_t launch_w4_quantize(const W4Layout &l, int experts, const float *B, int64_t ldb,
                              int64_t strideb, unsigned char *packed, hipStream_t s);
hipError_t launch_w4_unpack(const W4Layout &l, int experts, const unsigned char *packed, float *B,
                            int64_t ldb, int64_t strideb, hipStream_t s);
hipError_t launch_w4(const W4Layout &l, const W4Problem &p, hipStream_t s);

}  // namespace sgemm
