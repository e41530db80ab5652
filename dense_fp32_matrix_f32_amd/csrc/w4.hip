// w4.hip -- fp32 rows times a matrix of 4-bit weights.
//
//     C[i][n] = sum over groups g of s[g][n] * sum over k in g of A[i][k] * (q[k][n] - z[g][n])
//
// With few rows the bytes of the codes are the floor, so what is spent on a code
// besides its load has to stay below the time of that load: at 8 TB/s a CU gets
// about 26 codes a cycle, and its vector units do 64 operations a cycle.  The inner
// sums therefore run on the bf16 matrix cores, without any rounding of the inputs:
//   * a code 0 .. 15 is exact in bf16.  A byte 0 .. 15 read as an fp8 (e4m3) number
//     is that integer times 2^-9 (its denormals and first binade are one linear
//     run), so the byte pairs of a word become bf16 pairs by the conversion
//     instruction with scale 2^9: seven vector operations for eight codes;
//   * A[i][k] is cut into three bf16 parts that add up to it exactly (each part the
//     truncation of what is left, 8 bits at a time).  The parts of a row are rows of
//     their own in the matrix instruction: five rows of A fill one instruction of 16;
//   * z enters as z times the sum of A[i][k] over the group, which one more matrix
//     instruction with a matrix of ones forms in the registers' own layout.
// Products of parts and codes are exact in fp32 and are added in fp32; each group's
// sum is then scaled and added to the total in fp32.
//
// A work-group computes MR rows by CT strips of 16 columns over all k: its eight
// waves take the blocks of 128 k in turn (a block of a strip is one contiguous
// record, see w4.h), each with its own part of LDS for the parts of A, so no wave
// waits for another until the sums of the eight are added at the end, in a fixed
// order.
#include "groups.h"
#include "w4.h"

namespace sgemm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;

// Four vectors of bf16 pairs.
union Frag {
    bf16x8 v;
    bf16x2 pair[4];
    unsigned word[4];
};

// The eight codes of a word as bf16 integers.
__device__ __forceinline__ bf16x8 codes_of(unsigned w) {
    const unsigned lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    Frag f;
    f.pair[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    f.pair[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    f.pair[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    f.pair[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return f.v;
}

__device__ __forceinline__ unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }

// The upper halves of two floats as a bf16 pair.
__device__ __forceinline__ unsigned upper(float a, float b) {
    return __builtin_amdgcn_perm(bits(b), bits(a), 0x07060302u);
}

// What is left of x below its upper 16 bits (exact).
__device__ __forceinline__ float lower(float x) {
    return x - __builtin_bit_cast(float, bits(x) & 0xFFFF0000u);
}

// Writes by some lanes of a wave are read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// XV float4 vectors of A per lane and block: 2*XV rows (the last one odd at most);
// RT matrix-instruction rows of 16 hold the three parts of MR rows.
template <int XV>
struct Rows {
    static constexpr int MR = XV == 1 ? 2 : XV == 3 ? 5 : XV == 5 ? 10 : 16;
    static constexpr int RT = (3 * MR + 15) / 16;
};

template <int XV, int CT, int PARTS, int D>
__global__ __launch_bounds__(kWaves * 64) void w4_kernel(W4Layout l, W4Problem p, int row_blocks) {
    constexpr int MR = Rows<XV>::MR, RT = Rows<XV>::RT;
    constexpr int RP = 16 * RT + 1;   // 16-byte slots of one run of 8 k in LDS
    constexpr int STEPS = 4 / PARTS;  // matrix instructions of 32 k under one scale
    constexpr int COLS = kW4Cols * CT;
    constexpr int XS = 16 * RP * 16;                        // bytes of a wave's parts of A
    constexpr int RED = 16 * RT * (COLS + 1) * 4;           // bytes of a wave's sums
    __shared__ __attribute__((aligned(16))) unsigned char lds[kWaves * (XS > RED ? XS : RED)];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    // row blocks of one strip follow each other: they share its weights in one L2
    const int strip0 = id / row_blocks * CT;
    int expert = 0, first = id % row_blocks * MR, end = p.rows;
    if (p.offsets != nullptr &&
        !find_block(p.offsets, p.experts, p.rows, MR, id % row_blocks, &expert, &first, &end))
        return;
    const int rows = min(MR, end - first);

    const unsigned char *strip[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        strip[c] = p.packed + expert * l.expert_bytes +
                   min(strip0 + c, l.strips - 1) * l.strip_bytes;
    const float *arow[XV];
#pragma unroll
    for (int i = 0; i < XV; ++i)
        arow[i] = p.A + (int64_t)(first + min(2 * i + (lane >> 5), rows - 1)) * p.lda +
                  4 * (lane & 31);

    // One block of 128 k in registers: the loads of D blocks are in flight.
    struct Block {
        uint4 codes[CT];
        unsigned scale[CT][PARTS];
        unsigned zero[CT][PARTS];
        f32x4 x[XV];
    };
    auto load = [&](Block &b, int at) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const unsigned char *rec = strip[c] + (int64_t)at * l.record;
            b.codes[c] = *(const uint4 *)(rec + 16 * lane);
            const unsigned char *s = rec + kW4Codes;
#pragma unroll
            for (int t = 0; t < PARTS; ++t) {
                const int col = t * kW4Cols + (lane & 15);
                if (l.scale_size == 4) {
                    b.scale[c][t] = *(const unsigned *)(s + 4 * col);
                } else {
                    b.scale[c][t] = *(const unsigned short *)(s + 2 * col);
                }
                b.zero[c][t] = l.zeros ? s[PARTS * kW4Cols * l.scale_size + col] : 8;
            }
        }
        const int k = at * kW4Block;
        if (k + kW4Block <= l.K) {
#pragma unroll
            for (int i = 0; i < XV; ++i) __builtin_memcpy(&b.x[i], arow[i] + k, 16);
        } else {
            const int left = l.K - k - 4 * (lane & 31);
#pragma unroll
            for (int i = 0; i < XV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) b.x[i][e] = e < left ? arow[i][k + e] : 0.0f;
        }
    };

    unsigned char *xs = lds + wave * XS;
    // place of this lane's four k of row 2i + lane/32 (part 0); of its operand
    unsigned char *put = xs + (((lane & 31) >> 1) * RP + 3 * (lane >> 5)) * 16 + (lane & 1) * 8;
    const unsigned char *get = xs + ((lane >> 4) * RP + (lane & 15)) * 16;

    f32x4 total[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) total[r][c] = f32x4{};

    const Frag ones{.word = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};

    auto process = [&](const Block &b) {
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            if (2 * i + 1 >= MR && (lane >> 5)) continue;
            const f32x4 x = b.x[i];
            const f32x4 y = {lower(x[0]), lower(x[1]), lower(x[2]), lower(x[3])};
            const f32x4 z = {lower(y[0]), lower(y[1]), lower(y[2]), lower(y[3])};
            *(uint2 *)(put + 96 * i) = uint2{upper(x[0], x[1]), upper(x[2], x[3])};
            *(uint2 *)(put + 96 * i + 16) = uint2{upper(y[0], y[1]), upper(y[2], y[3])};
            *(uint2 *)(put + 96 * i + 32) = uint2{upper(z[0], z[1]), upper(z[2], z[3])};
        }
        wave_sync();
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
            f32x4 sum[RT][CT], sum_x[RT];
#pragma unroll
            for (int u = 0; u < STEPS; ++u) {
                const int j = t * STEPS + u;
                bf16x8 a[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    a[r] = *(const bf16x8 *)(get + (4 * j * RP + 16 * r) * 16);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    sum_x[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        a[r], ones.v, u ? sum_x[r] : f32x4{}, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const unsigned w = j == 0   ? b.codes[c].x
                                       : j == 1 ? b.codes[c].y
                                       : j == 2 ? b.codes[c].z
                                                : b.codes[c].w;
                    const bf16x8 q = codes_of(w);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        sum[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            a[r], q, u ? sum[r][c] : f32x4{}, 0, 0, 0);
                }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float s = l.scale_type == W4_F32 ? __builtin_bit_cast(float, b.scale[c][t])
                                : l.scale_type == W4_F16
                                    ? (float)__builtin_bit_cast(_Float16,
                                                                (unsigned short)b.scale[c][t])
                                    : __builtin_bit_cast(float, b.scale[c][t] << 16);
                const float z = (float)b.zero[c][t];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[r][c][e] =
                            fmaf(s, fmaf(-z, sum_x[r][e], sum[r][c][e]), total[r][c][e]);
            }
        }
        wave_sync();
    };

    // Blocks wave, wave + 8, ...: the loads of the next D are always issued before
    // one is used; past the last block they repeat it.
    const int n = (l.blocks - wave + kWaves - 1) / kWaves;
    if (n > 0) {
        Block b[D];
#pragma unroll
        for (int u = 0; u < D; ++u) load(b[u], wave + min(u, n - 1) * kWaves);
        int i = 0;
        for (; i + D < n; i += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                process(b[u]);
                load(b[u], wave + min(i + u + D, n - 1) * kWaves);
            }
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (i + u < n) process(b[u]);
    }

    // Add the waves' sums and the parts' rows, in the order of the parts and waves.
    __syncthreads();
    float *red = (float *)lds;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wave * 16 * RT + 16 * r + 4 * (lane >> 4) + e) * (COLS + 1) + 16 * c +
                    (lane & 15)] = total[r][c][e];
    __syncthreads();
    for (int o = threadIdx.x; o < rows * COLS; o += kWaves * 64) {
        const int m = o / COLS, col = o % COLS, n_at = strip0 * kW4Cols + col;
        if (n_at >= l.N) continue;
        float sum = 0.0f;
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                sum += red[(w * 16 * RT + 3 * m + part) * (COLS + 1) + col];
        p.C[(int64_t)(first + m) * p.ldc + n_at] = sum;
    }
}

template <int XV, int CT, int D>
hipError_t launch_rows(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    constexpr int MR = Rows<XV>::MR;
    const int64_t row_blocks = p.offsets != nullptr ? most_blocks(p.rows, p.experts, MR)
                                                    : ((int64_t)p.rows + MR - 1) / MR;
    const int64_t groups = ((int64_t)l.strips + CT - 1) / CT * row_blocks;
    if (groups > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)groups), block(kWaves * 64);
    switch (l.parts) {
    case 4: return launch(w4_kernel<XV, CT, 4, D>, grid, block, 0, s, l, p, (int)row_blocks);
    case 2: return launch(w4_kernel<XV, CT, 2, D>, grid, block, 0, s, l, p, (int)row_blocks);
    default: return launch(w4_kernel<XV, CT, 1, D>, grid, block, 0, s, l, p, (int)row_blocks);
    }
}

}  // namespace

hipError_t launch_w4(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    // rows that share a reading of the weights, where each expert has a like number
    const int64_t each = p.offsets != nullptr ? ((int64_t)p.rows + p.experts - 1) / p.experts : p.rows;
    if (each <= 2) return launch_rows<1, 1, 4>(l, p, s);
    if (each <= 5) return launch_rows<3, 1, 4>(l, p, s);
    if (each <= 10) return launch_rows<5, 1, 2>(l, p, s);
    // more rows than one block: the work of cutting A into parts is shared by four strips
    if (each <= 32) return launch_rows<8, 1, 2>(l, p, s);
    return launch_rows<8, 4, 2>(l, p, s);
}

}  // namespace sgemm
