// f8.h -- how matrices in 8-bit floating point are laid out on the device, shared by the
// kernels that write them and the products.
//
// An operand of a product is `rows` vectors over k (rows of A, or columns of B), cut into
// blocks of 128 k.  Block b of all rows is one plane, rows x 128 bytes, so the 16 rows of a
// matrix instruction are 2048 bytes side by side whatever row they begin at.  The 16-byte
// chunk c of a row (k = 16c .. 16c+15 of the block) is at place c ^ (row / 2) % 8: copied
// into LDS as it is, the 16 lanes that a 16-byte read serves at once (16 rows, one chunk)
// meet all 64 banks once, at any first row (in the order of k they would meet eight).
// What a block lacks of 128 k holds zeros.
//
// Scales.  Rows that are made here have a power of two for each row and block, kept as its
// biased exponent (a byte, 2^(byte - 127)): the four bytes of blocks 4t .. 4t+3 of a row are
// one word of [t][row].  Weights have an fp32 scale for each 128 x 128, [block of k][block
// of n], after the planes of an expert, whose rows are padded to 16.
#pragma once

#include "internal.h"

namespace sgemm {

constexpr int kF8Block = 128;

enum { F8_E4M3 = 0, F8_E5M2 = 1 };                  // codes, as the matrix instructions number them
enum { F8_IN_F32 = 0, F8_IN_BF16 = 1, F8_IN_ROWS = 2 };
enum { F8_SCALE_F32 = 0, F8_SCALE_E8M0 = 1 };

inline int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

// Weights: one expert's planes, then its scales, in bytes (a multiple of 16).
struct F8Weights {
    int64_t rows;         // N rounded up to 16
    int64_t blocks, cols; // blocks of k, blocks of n
    int64_t planes;       // bytes of the planes
    int64_t bytes;        // of an expert
};

inline F8Weights f8_weights(int64_t N, int64_t K) {
    F8Weights w;
    w.rows = (N + 15) / 16 * 16;
    w.blocks = f8_blocks(K);
    w.cols = f8_blocks(N);
    w.planes = w.blocks * w.rows * kF8Block;
    w.bytes = w.planes + (w.blocks * w.cols * 4 + 15) / 16 * 16;
    return w;
}

// Rows: planes, then words of four scales.
inline int64_t f8_row_planes(int64_t rows, int64_t blocks) { return blocks * rows * kF8Block; }
inline __int128 f8_rows_bytes(int64_t rows, int64_t blocks) {
    return (__int128)rows * blocks * kF8Block + (__int128)((blocks + 3) / 4) * rows * 4;
}

// Place of chunk c of a row, in bytes from the row's 128.
__host__ __device__ constexpr int f8_place(int chunk, int row) {
    return (chunk ^ (row >> 1 & 7)) * 16;
}

// The biased exponent of the smallest power of two s for which `most` / s is within the
// codes' largest number, 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2): the exponent of `most`
// less 8 or 15, one more if its fraction is above 1.75.  At least 2^-124 (2^-117), so that
// the smallest code stands for bf16's smallest number, 2^-133.  1 / s is exact, and so is x / s.
__device__ __forceinline__ int f8_scale_byte(float most, int type) {
    if (most == 0.0f) return 127;
    const int e = (int)((__builtin_bit_cast(unsigned, most) + 0x1FFFFFu) >> 23);
    return type == F8_E4M3 ? max(3, e - 8) : max(10, e - 15);
}
__device__ __forceinline__ float f8_exp2(int biased) {
    return __builtin_bit_cast(float, biased << 23);
}
// An fp32 scale as the power of two that goes into the codes' conversion and the rest of it, 1 to 2
// in size, that meets the fp32 sums of a block: these are then no larger than what they add to the
// result (sums of bare codes, up to 448 times the rows, overflowed from rows of 6e33 on).  Of the
// power the conversion reads the exponent's bits: none count as 2^-127, with a rest below 1 and
// down to zero, and all of them as NaN.
struct F8Scale {
    float power, rest;
};
__device__ __forceinline__ F8Scale f8_split(float s) {
    const unsigned bits = __builtin_bit_cast(unsigned, s);
    const float one = __builtin_bit_cast(float, (bits & 0x807FFFFFu) | 0x3F800000u);
    return {__builtin_bit_cast(float, bits & 0x7F800000u),
            (bits & 0x7F800000u) == 0 ? s * f8_exp2(254) : one};
}

// A scale that all lanes share, in a vector register until here.  The compiler would read it into a
// scalar one for f8_split(), next to its load, and wait there for every load before it (256 x
// 256 tiles 238 instead of 219 us).
__device__ __forceinline__ float f8_here(float s) {
    asm volatile("" : "+v"(s));
    return s;
}

// 2^(127 - byte), byte in 3 .. 247
__device__ __forceinline__ float f8_inverse(int byte) { return f8_exp2(254 - byte); }

// |x| as it counts for a scale: numbers that are none (NaN, infinities) count for nothing,
// their own codes are NaN.
__device__ __forceinline__ float f8_size(float x) {
    const float a = __builtin_fabsf(x);
    return a <= __FLT_MAX__ ? a : 0.0f;
}

// Four codes of x * inv (to nearest, ties to even); infinities become NaN.
template <int TYPE>
__device__ __forceinline__ unsigned f8_codes(float x0, float x1, float x2, float x3, float inv) {
    int r = 0;
    if constexpr (TYPE == F8_E4M3) {
        // the instruction's largest number stands for infinities too: x - x is NaN for them
        // and 0 for numbers
        r = __builtin_amdgcn_cvt_pk_fp8_f32(x0 * inv + (x0 - x0), x1 * inv + (x1 - x1), r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(x2 * inv + (x2 - x2), x3 * inv + (x3 - x3), r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(x0 * inv + (x0 - x0), x1 * inv + (x1 - x1), r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(x2 * inv + (x2 - x2), x3 * inv + (x3 - x3), r, true);
    }
    return (unsigned)r;
}

// Sixteen values of a row from x on (`left` of them inside it, the others zero).
template <class T>
__device__ __forceinline__ void f8_load16(const T *x, int left, float (&v)[16]) {
    if (left >= 16) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) __builtin_memcpy(&v[4 * q], x + 4 * q, 16);
        } else {
            unsigned w[8];
            __builtin_memcpy(w, x, 16);
            __builtin_memcpy(w + 4, x + 8, 16);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[2 * q] = __builtin_bit_cast(float, w[q] << 16);
                v[2 * q + 1] = __builtin_bit_cast(float, w[q] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = q < left ? (float)x[q] : 0.0f;
    }
}

// bf16 numbers, converted as they are read.
struct Bf16 {
    unsigned short bits;
    __device__ operator float() const { return __builtin_bit_cast(float, (unsigned)bits << 16); }
};

template <int CTRL>
__device__ __forceinline__ float f8_lane(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                                 0xf, 0xf, true));
}

// The largest over 8 neighbouring lanes.
__device__ __forceinline__ float f8_max8(float x) {
    x = fmaxf(x, f8_lane<0xB1>(x));
    x = fmaxf(x, f8_lane<0x4E>(x));
    return fmaxf(x, f8_lane<0x141>(x));
}

// The codes of 16 of the 128 numbers of a row and block, which eight neighbouring lanes
// hold, and the scale's byte.
template <int TYPE>
__device__ __forceinline__ uint4 f8_chunk(const float (&v)[16], unsigned *byte) {
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) most = fmaxf(most, f8_size(v[e]));
    *byte = f8_scale_byte(f8_max8(most), TYPE);
    const float inv = f8_inverse(*byte);
    return uint4{f8_codes<TYPE>(v[0], v[1], v[2], v[3], inv),
                 f8_codes<TYPE>(v[4], v[5], v[6], v[7], inv),
                 f8_codes<TYPE>(v[8], v[9], v[10], v[11], inv),
                 f8_codes<TYPE>(v[12], v[13], v[14], v[15], inv)};
}

// Rows of numbers to be put into 8 bits.
struct F8RowsProblem {
    int rows, K;
    const void *A;
    int64_t lda;
    int in, type;
    unsigned char *q;
};
hipError_t launch_f8_rows(const F8RowsProblem &p, hipStream_t s);

// The columns of rows x width numbers, in blocks of 128 rows of an expert: an operand whose
// rows are the columns and whose blocks are the experts' blocks, one expert after another
// (`blocks`: the most there can be).
struct F8ColumnsProblem {
    int rows, width, experts;
    const int *offsets;
    const void *A;
    int64_t lda;
    int in, type;
    int64_t blocks;
    unsigned char *q;
};
hipError_t launch_f8_columns(const F8ColumnsProblem &p, hipStream_t s);

// Matrices R x C (row-major, `stride` apart) as an operand of rows c over r (`down`) and one
// of rows r over c (`along`); either may be NULL.  With codes, those and their scales are
// taken over, else they are formed from the fp32 numbers.
struct F8MatrixProblem {
    int experts, R, C;
    const void *source;       // fp32, or codes
    int64_t ld, stride;
    const void *scales;       // of codes: experts x blocks of R x blocks of C
    int scale_type;
    unsigned char *down, *along;
};
hipError_t launch_f8_quantize(const F8MatrixProblem &p, hipStream_t s);
hipError_t launch_f8_pack(const F8MatrixProblem &p, hipStream_t s);
hipError_t launch_f8_unpack(int experts, int N, int K, const unsigned char *packed, float *B,
                            int64_t ldb, int64_t strideb, hipStream_t s);

// Products of rows (numbers, or an operand made before) with weights.
struct F8Problem {
    int rows, N, K, experts;
    const int *offsets;       // NULL: one matrix
    const void *A;
    int64_t lda;
    int in, type;
    const unsigned char *packed;
    int scale_type;
    void *C;
    int64_t ldc;
    bool bf16;                // C is bf16, else fp32
    unsigned char *workspace;
    bool check;               // only whether one launch holds it
};
size_t f8_workspace(int rows, int N, int K, int experts, bool by_expert);
hipError_t launch_f8(const F8Problem &p, hipStream_t s);

// C_e (M x N) = alpha * A_e^T * D_e + beta * C_e over each expert's rows, both in 8 bits
// along their columns.
struct F8TaProblem {
    int rows, M, N, experts;
    const int *offsets;
    const void *A;
    int64_t lda;
    int a_in, a_type;
    const void *D;
    int64_t ldd;
    int d_in, d_type;
    float alpha, beta;
    float *C;
    int64_t ldc, stridec;
    unsigned char *workspace;
    bool check;
};
__int128 f8_ta_workspace(int rows, int M, int N, int experts);
hipError_t launch_f8_ta(const F8TaProblem &p, hipStream_t s);

}  // namespace sgemm
