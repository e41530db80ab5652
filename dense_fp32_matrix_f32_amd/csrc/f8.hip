// f8.hip -- products of operands in 8-bit floating point with a scale for each block of 128 k.
//
//     C[m][n] = sum over blocks b of sx[b][m] * sw[b][n] * sum over k in b of x[m][k] * w[n][k]
//
// (layout and scales in f8.h).  Sums are kept in fp32.  The 8-bit matrix instructions of gfx950 do
// not: they form 128 products of an element at three times the rate of the bf16 ones (3.8 against
// 1.1 PFLOP/s without loads), but add each eight of them with about 14 bits below the largest,
// so results are 1.5e-5 to 4e-5 off in the 2-norm on random data and have no right digit where
// large terms cancel.  The codes become bf16 numbers instead, which hold every code and power
// of two exactly, and the bf16 instructions add their products in fp32 (5e-8).  The powers of two
// go into the codes' conversion.  So does that of a general fp32 scale of the weights, and the rest
// of it meets a block's fp32 sums as they are added to the total (f8_split()).
//
// The weights are the first operand of the matrix instructions, so a lane holds four
// neighbouring columns of a row of C.
#include <type_traits>

#include "f8.h"
#include "groups.h"

namespace sgemm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// How the scales of the first operand (the weights) are kept.
enum { W_F32, W_POW2, W_ROWS };

// One operand: planes of `rows` x 128 bytes, and its scales.
struct Side {
    const unsigned char *codes;
    const unsigned char *scales;
    int64_t rows;
};

struct F8Args {
    Side x, w;
    int64_t expert;      // bytes between experts' weights (and their scales)
    int64_t scale_cols;  // blocks of n
    int blocks;          // of k (of an expert's weights)
    int M, N, experts;
    const int *offsets;
    void *C;
    int64_t ldc, stridec;
    float alpha, beta;
    bool wide;           // four columns of C can be stored at once
};

// Eight codes as bf16 numbers times the power of two s.
template <int TYPE>
__device__ __forceinline__ bf16x8 to_bf16(unsigned lo, unsigned hi, float s) {
    union {
        bf16x8 v;
        bf16x2 p[4];
    } f;
    if constexpr (TYPE == F8_E4M3) {
        f.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
        f.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
        f.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
        f.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
    } else {
        f.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, s, false);
        f.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, s, true);
        f.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, s, false);
        f.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, s, true);
    }
    return f.v;
}

// A lane's 32 codes of a row and block: chunks g and g + 4, g = lane / 16.
union Codes {
    uint4 half[2];
    unsigned word[8];
    __device__ __forceinline__ void load(const unsigned char *p, unsigned at) {
        half[0] = *(const uint4 *)(p + at);
        half[1] = *(const uint4 *)(p + (at ^ 64));
    }
    template <int TYPE>
    __device__ __forceinline__ void widen(float s, bf16x8 (&out)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = to_bf16<TYPE>(word[2 * j], word[2 * j + 1], s);
    }
};

__device__ __forceinline__ void store4(const F8Args &p, float *C, f32x4 v, int64_t at, int left) {
    float *c = C + at;
    if (p.alpha != 1.0f || p.beta != 0.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) v[e] = epilogue(v[e], p.alpha, p.beta, c + e);
    }
    if (p.wide && left >= 4) {
        *(f32x4 *)c = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) c[e] = v[e];
    }
}
__device__ __forceinline__ void store4(const F8Args &p, __bf16 *C, f32x4 v, int64_t at, int left) {
    // (as a vector: taken apart, the totals of 256 x 256 no longer fit the registers)
    const bf16x4 r = __builtin_convertvector(v, bf16x4);
    if (p.wide && left >= 4) {
        *(bf16x4 *)(C + at) = r;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) C[at + e] = r[e];
    }
}

// ---------------------------------------------------------------------------
// Many rows: a work-group forms BM rows by BN columns of C, each wave TM x TN tiles of 16 x
// 16.  A block of 128 k of both operands is copied straight into LDS while the one before
// is multiplied: two stages and one barrier a block.
template <int WM_, int WN_, int TM_, int TN_>
struct F8Tile {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
    static constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN, WAVES = WM * WN;
    static constexpr int THREADS = 64 * WAVES, CODES = (BM + BN) * kF8Block;
    static constexpr int STAGE = CODES + (BM + BN) * 4;  // with a word of scales a row
    static constexpr int UNITS = (BM + BN) / 8 / WAVES;  // copies of 8 rows x 128 bytes a wave makes
    static constexpr int X_UNITS = BM / 8 / WAVES;  // of them of x, then those of w
    static_assert(BM == BN && BM % (8 * WAVES) == 0 && BM % 64 == 0 && BM / 64 <= WAVES,
                  "whole copies");
};

typedef unsigned char __attribute__((address_space(3))) *LdsBytes;

template <class T, class OUT, int WS, int WT, int XT>
__device__ __forceinline__ void f8_tile(const F8Args &p, unsigned char *stage0,
                                        unsigned char *stage1, int expert, int first, int rows,
                                        int n0, int block0, int blocks, int64_t c0) {
    constexpr int TM = T::TM, TN = T::TN;
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;

    // Copies: unit u of this wave is 8 rows of x or of w, 1024 bytes side by side in LDS; then
    // the words of scales, 64 rows a copy.  They go through buffer resources that end with the
    // rows there are, so a block at the edge reads nothing past them.  A copy's whole place is its
    // vector offset: the range check is sure to count that one, the scalar one it leaves out or
    // takes from the size, which wraps where there are fewer rows than it steps over.
    const int64_t x_plane = p.x.rows * kF8Block, w_plane = p.w.rows * kF8Block;
    const unsigned char *xb = p.x.codes + block0 * x_plane + (int64_t)first * kF8Block;
    const unsigned char *wb = p.w.codes + expert * p.expert +
                              (WS == W_ROWS ? block0 : 0) * w_plane + (int64_t)n0 * kF8Block;
    const int w_rows = (int)min((int64_t)T::BN, p.w.rows - n0);
    auto resource = [](const unsigned char *base, int bytes) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, bytes, 0x00020000);
    };
    auto copy = [&](unsigned char *stage, int b) {
        const auto xr = resource(xb, rows * kF8Block), wr = resource(wb, w_rows * kF8Block);
#pragma unroll
        for (int u = 0; u < T::UNITS; ++u) {
            const int unit = wave + u * T::WAVES;
            const LdsBytes to = (LdsBytes)(stage + unit * 1024);
            const int at = (wave + u % T::X_UNITS * T::WAVES) * 1024 + lane * 16;
            if (u < T::X_UNITS)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, to, 16, at, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, at, 0, 0, 0);
        }
        const int word = (block0 + b) >> 2;
        if (wave < T::BM / 64) {
            const auto r = resource(p.x.scales + ((int64_t)word * p.x.rows + first) * 4, rows * 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsBytes)(stage + T::CODES + wave * 256), 4,
                                                     wave * 256 + lane * 4, 0, 0, 0);
        }
        if constexpr (WS == W_ROWS) {
            if (wave < T::BN / 64) {
                const auto r =
                    resource(p.w.scales + ((int64_t)word * p.w.rows + n0) * 4, w_rows * 4);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    r, (LdsBytes)(stage + T::CODES + T::BM * 4 + wave * 256), 4,
                    wave * 256 + lane * 4, 0, 0, 0);
            }
        }
        xb += x_plane;
        wb += w_plane;
    };

    // this lane's rows: x tile t is row 16t further, w tile t column 16t
    const int xrow = wm * 16 * TM + i, wrow = wn * 16 * TN + i;
    const unsigned x_at = xrow * kF8Block + f8_place(g, first + i);
    const unsigned w_at = (T::BM + wrow) * kF8Block + f8_place(g, i);
    const float *w_scale = (const float *)(p.w.scales + expert * p.expert) +
                           min((n0 + wn * 16 * TN) / kF8Block, (int)p.scale_cols - 1);
    float sw = 1.0f, sw_next = 1.0f;  // the scale of a block, loaded a block ahead

    f32x4 acc[TM][TN];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) acc[tm][tn] = f32x4{};

    auto multiply = [&](const unsigned char *s, int b) {
        const unsigned char *xs = s + T::CODES + xrow * 4 + ((block0 + b) & 3);
        const unsigned char *ws = s + T::CODES + (T::BM + wrow) * 4 + ((block0 + b) & 3);
        // (here a scalar: 233 instead of 234.5 us for 4096 x 4096 x 8192 in bf16)
        const F8Scale scale =
            WS == W_F32 ? f8_split(__builtin_bit_cast(
                              float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, sw))))
                        : F8Scale{sw, 1.0f};
        bf16x8 w[TN][4];
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
            Codes c;
            c.load(s, w_at + tn * 16 * kF8Block);
            c.widen<WT>(WS == W_ROWS ? f8_exp2(ws[64 * tn]) : scale.power, w[tn]);
        }
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            Codes c;
            c.load(s, x_at + tm * 16 * kF8Block);
            bf16x8 x[4];
            c.widen<XT>(f8_exp2(xs[64 * tm]), x);
            f32x4 part[TN];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int tn = 0; tn < TN; ++tn) {
                    if constexpr (WS == W_F32)
                        part[tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            w[tn][j], x[j], j == 0 ? f32x4{} : part[tn], 0, 0, 0);
                    else
                        acc[tm][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            w[tn][j], x[j], acc[tm][tn], 0, 0, 0);
                }
            if constexpr (WS == W_F32) {
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[tm][tn][e] = fmaf(scale.rest, part[tn][e], acc[tm][tn][e]);
            }
        }
    };

    // Stages are arrays of their own: the compiler then sees that a block's reads do not meet
    // the copies in flight, and does not wait for those.
    auto step = [&](int b, unsigned char *now, unsigned char *next) {
        // the copies of this block have arrived, in all waves; the other stage is read no more
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
        sw = sw_next;
        if (b + 1 < blocks) {
            copy(next, b + 1);
            if constexpr (WS != W_ROWS) sw_next = w_scale[(b + 1) * p.scale_cols];
        }
        multiply(now, b);
    };
    if (blocks > 0) {
        copy(stage0, 0);
        if constexpr (WS != W_ROWS) sw_next = w_scale[0];
    }
    for (int b = 0; b < blocks; b += 2) {
        step(b, stage0, stage1);
        if (b + 1 < blocks) step(b + 1, stage1, stage0);
    }

    // a lane holds row i and columns 4g .. 4g+3 of each tile
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
        const int m = xrow + 16 * tm;
        if (m >= rows) continue;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
            const int n = n0 + wn * 16 * TN + 16 * tn + 4 * g;
            if (n < p.N)
                store4(p, (OUT *)p.C, acc[tm][tn], c0 + (int64_t)(first + m) * p.ldc + n, p.N - n);
        }
    }
}

// C rows = x rows times the weights of their expert.
template <class T, class OUT, int WS, int XT>
__global__ __launch_bounds__(T::THREADS) void f8_kernel(F8Args p, int tiles_n) {
    __shared__ __attribute__((aligned(16))) unsigned char stage0[T::STAGE];
    __shared__ __attribute__((aligned(16))) unsigned char stage1[T::STAGE];
    int tm, tn, expert = 0, first, end = p.M;
    if (p.offsets != nullptr) {
        // (offsets that are no running sum can give more blocks than were launched, or a
        // count that wrapped to a negative one)
        const int tiles_m = min(count_blocks(p.offsets, p.experts, p.M, AllBlocks{T::BM}),
                                (int)(gridDim.x / (unsigned)tiles_n));
        if ((int)blockIdx.x >= tiles_m * tiles_n) return;
        tile_order(blockIdx.x, tiles_m, tiles_n, 4, &tm, &tn);
        if (!find_block(p.offsets, p.experts, p.M, T::BM, tm, &expert, &first, &end)) return;
    } else {
        tile_order(blockIdx.x, gridDim.x / (unsigned)tiles_n, tiles_n, 4, &tm, &tn);
        first = tm * T::BM;
    }
    f8_tile<T, OUT, WS, F8_E4M3, XT>(p, stage0, stage1, expert, first, min(T::BM, end - first),
                                      tn * T::BN, 0, p.blocks, 0);
}

// C_e = the sum over the blocks of expert e's rows: operands whose rows are the columns of A
// and D.
template <class T, int WT, int XT>
__global__ __launch_bounds__(T::THREADS) void f8_ta_kernel(F8Args p, int rows, int tiles_m,
                                                          int tiles_n) {
    __shared__ __attribute__((aligned(16))) unsigned char stage0[T::STAGE];
    __shared__ __attribute__((aligned(16))) unsigned char stage1[T::STAGE];
    const int tiles = tiles_m * tiles_n;
    const int e = blockIdx.x / tiles;
    int block0 = 0, blocks = p.blocks;
    if (p.offsets != nullptr) {
        const int lo = clamp_row(p.offsets[e], rows);
        blocks = AllBlocks{kF8Block}(max(lo, clamp_row(p.offsets[e + 1], rows)) - lo);
        block0 = count_blocks(p.offsets, e, rows, AllBlocks{kF8Block});
        // (offsets that are no running sum: within the blocks that were made)
        block0 = max(0, min(block0, p.blocks));
        blocks = min(blocks, p.blocks - block0);
    }
    int tm, tn;
    tile_order(blockIdx.x % tiles, tiles_m, tiles_n, 4, &tm, &tn);
    const int first = tm * T::BM;
    f8_tile<T, float, W_ROWS, WT, XT>(p, stage0, stage1, 0, first, min(T::BM, p.M - first),
                                     tn * T::BN, block0, blocks, e * p.stridec);
}

// ---------------------------------------------------------------------------
// Few rows: bound by reading the weights once.  A work-group forms 16 RT rows by 16 CT
// columns; its eight waves take the blocks of 128 k in turn, operands go from memory to the
// registers without LDS, and the waves' sums are added at the end, in a fixed order.  The
// rows are codes that f8_rows_kernel has made; up to kFewRows come as numbers and are put
// into 8 bits by every work-group for itself, in LDS, while its first weights are on
// their way (the same codes).
struct FewArgs {
    F8Args a;
    const void *A;
    int64_t lda;
    int K;
};

constexpr int kFewWaves = 8, kFewRows = 4;
constexpr int kFewK = 8192;  // 33 KB of LDS for the codes of kFewRows rows

// IN: float, Bf16 (numbers) or void (codes).
template <class IN, int RT, int CT, int D, bool POW2, int XT, class OUT>
__global__ __launch_bounds__(64 * kFewWaves) void f8_few_kernel(FewArgs f, int row_blocks) {
    constexpr bool CODES = std::is_same<IN, void>::value;
    constexpr int W = kFewWaves, BM = CODES ? 16 * RT : kFewRows, BN = 16 * CT;
    static_assert(CODES || RT == 1, "one tile of rows");
    const F8Args &p = f.a;
    __shared__ float red[W][BM][BN + 4];
    extern __shared__ __attribute__((aligned(16))) unsigned char made[];
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // row blocks that read the same weights follow each other
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const unsigned row_block = id % (unsigned)row_blocks;
    const int n0 = id / (unsigned)row_blocks * BN;
    int expert = 0, first = row_block * BM, end = p.M;
    if (p.offsets != nullptr &&
        !find_block(p.offsets, p.experts, p.M, BM, row_block, &expert, &first, &end))
        return;
    const int rows = min(BM, end - first);

    const unsigned char *wp[CT];
    const float *sp[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int n = (int)min((int64_t)(n0 + 16 * c), p.w.rows - 16);
        wp[c] = p.w.codes + expert * p.expert + (int64_t)(n + i) * kF8Block + f8_place(g, i);
        sp[c] = (const float *)(p.w.scales + expert * p.expert) + n / kF8Block;
    }
    const int64_t w_plane = p.w.rows * kF8Block;
    // (place of chunk g + 4 = place of chunk g with 64 flipped)
    const int flip = (f8_place(g, i) & 64) ? -64 : 64;

    struct Block {
        uint4 w[CT][2];
        float s[CT];
        uint4 x[CODES ? RT : 1][2];
        unsigned xs[CODES ? RT : 1];
    };
    const int64_t x_plane = p.x.rows * kF8Block;
    int xr[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) xr[r] = first + min(16 * r + i, rows - 1);
    auto load = [&](Block &b, int block) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const unsigned char *w = wp[c] + block * w_plane;
            b.w[c][0] = *(const uint4 *)w;
            b.w[c][1] = *(const uint4 *)(w + flip);
            b.s[c] = sp[c][block * p.scale_cols];
        }
        if constexpr (CODES) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const unsigned char *x = p.x.codes + block * x_plane + (int64_t)xr[r] * kF8Block;
                const int at = f8_place(g, xr[r]);
                b.x[r][0] = *(const uint4 *)(x + at);
                b.x[r][1] = *(const uint4 *)(x + (at ^ 64));
                b.xs[r] = p.x.scales[((int64_t)(block >> 2) * p.x.rows + xr[r]) * 4 + (block & 3)];
            }
        }
    };

    f32x4 total[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) total[r][c] = f32x4{};

    auto process = [&](const Block &b, int block) {
        bf16x8 x[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            Codes c;
            unsigned byte;
            if constexpr (CODES) {
                c.half[0] = b.x[r][0];
                c.half[1] = b.x[r][1];
                byte = b.xs[r];
            } else {
                const int row = min(i, rows - 1);
                c.load(made, (block * BM + row) * kF8Block + f8_place(g, row));
                byte = made[p.blocks * BM * kF8Block + block * BM + row];
            }
            c.widen<XT>(f8_exp2(byte), x[r]);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            Codes codes;
            codes.half[0] = b.w[c][0];
            codes.half[1] = b.w[c][1];
            bf16x8 w[4];
            const F8Scale scale = POW2 ? F8Scale{b.s[c], 1.0f} : f8_split(f8_here(b.s[c]));
            codes.widen<F8_E4M3>(scale.power, w);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                f32x4 sum = POW2 ? total[r][c] : f32x4{};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], x[r][j], sum, 0, 0, 0);
                if constexpr (POW2) {
                    total[r][c] = sum;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[r][c][e] = fmaf(scale.rest, sum[e], total[r][c][e]);
                }
            }
        }
    };

    // Blocks wave, wave + W, ...: the loads of the next D are always issued before one is
    // used; past the last block they repeat it.
    // Numbers: eight lanes put the 128 of a row and block into 8 bits.  The first of them are
    // asked for before the first weights, since loads arrive in the order they were made in.
    const int n = (p.blocks - wave + W - 1) / W, tasks = CODES ? 0 : rows * p.blocks * 8;
    auto numbers = [&](int task, float(&v)[16]) {
        if constexpr (!CODES) {
            const int block = (task >> 3) % p.blocks, row = (task >> 3) / p.blocks;
            const int k = block * kF8Block + (task & 7) * 16;
            f8_load16((const IN *)f.A + (int64_t)(first + row) * f.lda + k, f.K - k, v);
        }
    };
    float v[16];
    if ((int)threadIdx.x < tasks) numbers(threadIdx.x, v);
    Block b[D];
    if (n > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) load(b[u], wave + min(u, n - 1) * W);
    }
    if constexpr (!CODES) {
        for (int task = threadIdx.x; task < tasks; task += 64 * W) {
            if (task >= 64 * W) numbers(task, v);
            const int chunk = task & 7, block = (task >> 3) % p.blocks, row = (task >> 3) / p.blocks;
            unsigned byte;
            const uint4 codes = f8_chunk<XT>(v, &byte);
            *(uint4 *)(made + (block * BM + row) * kF8Block + f8_place(chunk, row)) = codes;
            if (chunk == 0) made[p.blocks * BM * kF8Block + block * BM + row] = (unsigned char)byte;
        }
        __syncthreads();
    }
    if (n > 0) {
        int t = 0;
        for (; t + D < n; t += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                process(b[u], wave + (t + u) * W);
                load(b[u], wave + min(t + u + D, n - 1) * W);
            }
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (t + u < n) process(b[u], wave + (t + u) * W);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (16 * r + i < BM) *(f32x4 *)&red[wave][16 * r + i][16 * c + 4 * g] = total[r][c];
    __syncthreads();
    for (int o = threadIdx.x; o < rows * (BN / 4); o += 64 * W) {
        const int m = o / (BN / 4), c = o % (BN / 4) * 4, at = n0 + c;
        if (at >= p.N) continue;
        f32x4 sum = *(const f32x4 *)&red[0][m][c];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += *(const f32x4 *)&red[w][m][c];
        store4(p, (OUT *)p.C, sum, (int64_t)(first + m) * p.ldc + at, p.N - at);
    }
}

// K == 0: zeros in the experts' rows.
template <class OUT>
__global__ __launch_bounds__(256) void f8_zero_kernel(F8Args p) {
    const int experts = p.offsets != nullptr ? p.experts : 1;
    for (int e = 0; e < experts; ++e) {
        const int lo = p.offsets != nullptr ? clamp_row(p.offsets[e], p.M) : 0;
        const int hi = p.offsets != nullptr ? max(lo, clamp_row(p.offsets[e + 1], p.M)) : p.M;
        for (int64_t i = (int64_t)lo + blockIdx.x; i < hi; i += gridDim.x)
            for (int64_t n = threadIdx.x; n < p.N; n += 256) ((OUT *)p.C)[i * p.ldc + n] = (OUT)0.0f;
    }
}

// ---------------------------------------------------------------------------

bool can_store4(const void *C, int64_t ldc, int size) {
    return ((uintptr_t)C & (4 * size - 1)) == 0 && ldc % 4 == 0;
}

int64_t row_blocks(const F8Problem &p, int bm) {
    return p.offsets != nullptr ? most_blocks(p.rows, p.experts, bm)
                                : ((int64_t)p.rows + bm - 1) / bm;
}

template <class IN, int RT, int CT, int D, int XT, class OUT>
hipError_t launch_few_as(const F8Problem &p, const FewArgs &f, hipStream_t s) {
    constexpr bool CODES = std::is_same<IN, void>::value;
    const int64_t rb = row_blocks(p, CODES ? 16 * RT : kFewRows);
    const int64_t groups = ((int64_t)p.N + 16 * CT - 1) / (16 * CT) * rb;
    if (groups > most_groups(64 * kFewWaves)) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    const dim3 grid((unsigned)groups), block(64 * kFewWaves);
    const size_t lds = CODES ? 0 : (size_t)f.a.blocks * kFewRows * (kF8Block + 1);
    if (p.scale_type == F8_SCALE_E8M0)
        return launch(f8_few_kernel<IN, RT, CT, D, true, XT, OUT>, grid, block, lds, s, f, (int)rb);
    return launch(f8_few_kernel<IN, RT, CT, D, false, XT, OUT>, grid, block, lds, s, f, (int)rb);
}

template <class T, class OUT, int WS, int XT>
hipError_t launch_many_with(const F8Problem &p, const F8Args &a, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + T::BN - 1) / T::BN;
    const int64_t groups = row_blocks(p, T::BM) * tiles_n;
    if (groups > most_groups(T::THREADS)) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    return launch(f8_kernel<T, OUT, WS, XT>, dim3((unsigned)groups), dim3(T::THREADS), 0, s, a,
                  (int)tiles_n);
}

template <class T, int XT, class OUT>
hipError_t launch_many_as(const F8Problem &p, const F8Args &a, hipStream_t s) {
    return p.scale_type == F8_SCALE_E8M0 ? launch_many_with<T, OUT, W_POW2, XT>(p, a, s)
                                         : launch_many_with<T, OUT, W_F32, XT>(p, a, s);
}

using Tile64 = F8Tile<2, 2, 2, 2>;    // 64 x 64, four waves
using Tile128 = F8Tile<2, 2, 4, 4>;   // 128 x 128, four waves
using Tile256 = F8Tile<2, 4, 8, 4>;   // 256 x 256, eight waves

// Rows that an expert has on average.
int64_t rows_each(int rows, int experts, bool by_expert) {
    return by_expert ? ((int64_t)rows + experts - 1) / experts : rows;
}

// Tiles of C for many rows: the larger ones read each operand less often from LDS and memory,
// the smaller ones fill the CUs with fewer rows and waste less of an expert's last one.  Both
// types of results are summed alike and differ in their stores only.  Times in us with fp32 / power
// of two scales:
//   rows  N x K, result             64 x 64    128 x 128   256 x 256
//    512  4096 x 4096, fp32          25 / 21     40 / 35    104 / 85
//   1024  4096 x 4096, fp32          47 / 40     47 / 43    107 / 89
//   4096  8192 x 4096, fp32         335 / 270   247 / 230   221 / 194
//   8192  8192 x 8192, fp32        1241 / 1075  944 / 851   852 / 734
//   2048 by expert, 8 x 4096 x 2048, fp32    50 / 44     52 / 47     61 / 52
//  16384 by expert, 8 x 2048 x 4096, fp32   345 / 296   272 / 247   320 / 270
//  16384 by expert, 8 x 4096 x 2048, fp32   372 / 319   288 / 252   298 / 257
//    512  4096 x 4096, bf16          29 / 23     47 / 38    107 / 90
//   1024  8192 x 4096, bf16          92 / 73     79 / 64    109 / 92
//   4096  8192 x 4096, bf16         322 / 270   261 / 221   219 / 190
//   8192  8192 x 8192, bf16        1220 / 1057  984 / 832   827 / 722
//   2048 by expert, 32 x 2048 x 1024, bf16   23 / 19     25 / 20     34 / 28
//  16384 by expert, 8 x 4096 x 2048, bf16   354 / 316   293 / 252   294 / 254
// (4096 rows of 8192 x 4096 are 228 us at the rate that a bf16 product of the library reaches, 1203
// TFLOP/s.)
template <int XT, class OUT>
hipError_t launch_many(const F8Problem &p, const F8Args &a, hipStream_t s) {
    const bool by_expert = p.offsets != nullptr;
    const int64_t each = rows_each(p.rows, p.experts, by_expert), cus = compute_units();
    auto tiles = [&](int64_t b) {
        return ((int64_t)p.N + b - 1) / b * ((each + b - 1) / b) * (by_expert ? p.experts : 1);
    };
    if (tiles(256) >= (by_expert ? 4 : 2) * cus) return launch_many_as<Tile256, XT, OUT>(p, a, s);
    if (tiles(128) >= cus && (!by_expert || each >= 512))
        return launch_many_as<Tile128, XT, OUT>(p, a, s);
    return launch_many_as<Tile64, XT, OUT>(p, a, s);
}

// The kernel for codes, by the rows that share a reading of the weights.  Times in us, back
// to back, random data, the weights of two or three calls in turn:
//   rows  N x K                  16 rows by 16, 32 columns   32 rows by 16, 32, 64   128 x 128
//    1    4096 x 4096                 4.6   5.3
//   16    4096 x 4096                 5.0   5.7
//   16    8192 x 8192                12.3  12.0
//   32    4096 x 4096                                         6.1   6.9   8.8
//   37    1023 x 4097                                         6.1   6.9   9.3
//   64    4096 x 4096                                        10.0   7.3   9.0          38
//   64    8192 x 8192                                        30.5  20.5  15.7          72
//  128    4096 x 4096                                        16.2  11.8   9.1          38
//  256    4096 x 4096                                        30.2  20.1  16.9          39
//    8 by expert, 64 x 2048 x 2048    7.8   7.8               8.8   8.2   8.7
//   48 by expert, 8 x 4096 x 2048    13.3  13.4              15.2  14.7  14.9
//  128 by expert, 8 x 4096 x 2048    17.9  15.0              16.8  15.2  15.2          22
//  256 by expert, 16 x 1024 x 2048   10.5   8.7              10.3   8.8   8.7          21
template <int XT, class OUT>
hipError_t launch_codes(const F8Problem &p, const FewArgs &f, hipStream_t s) {
    const int64_t each = rows_each(p.rows, p.experts, p.offsets != nullptr);
    const int64_t strips = ((int64_t)p.N + 15) / 16;
    if (each <= 16)
        return strips * row_blocks(p, 16) >= 512 ? launch_few_as<void, 1, 2, 1, XT, OUT>(p, f, s)
                                                 : launch_few_as<void, 1, 1, 1, XT, OUT>(p, f, s);
    if (each <= 256) {
        const int64_t groups = strips * row_blocks(p, 32);
        if (groups >= 1024) return launch_few_as<void, 2, 4, 1, XT, OUT>(p, f, s);
        if (groups >= 512) return launch_few_as<void, 2, 2, 1, XT, OUT>(p, f, s);
        return launch_few_as<void, 2, 1, 1, XT, OUT>(p, f, s);
    }
    return launch_many<XT, OUT>(p, f.a, s);
}

// Whether rows given as numbers are put into 8 bits by a kernel of its own.
bool rows_first(int rows, int K, int experts, bool by_expert) {
    return rows_each(rows, experts, by_expert) > kFewRows || K > kFewK;
}

template <int XT, class OUT>
hipError_t launch_product(const F8Problem &p, const FewArgs &f, hipStream_t s) {
    if (f.a.x.codes != nullptr) return launch_codes<XT, OUT>(p, f, s);
    return p.in == F8_IN_F32 ? launch_few_as<float, 1, 1, 2, XT, OUT>(p, f, s)
                             : launch_few_as<Bf16, 1, 1, 2, XT, OUT>(p, f, s);
}

}  // namespace

size_t f8_workspace(int rows, int N, int K, int experts, bool by_expert) {
    if (N == 0 || K == 0 || rows == 0 || experts == 0 || !rows_first(rows, K, experts, by_expert))
        return 0;
    const __int128 bytes = f8_rows_bytes(rows, f8_blocks(K));
    return bytes > ((__int128)1 << 62) ? SIZE_MAX : (size_t)bytes;
}

namespace {

// The rows into 8 bits, if they are not, and the product.
hipError_t run_f8(const F8Problem &p, hipStream_t s) {
    const F8Weights l = f8_weights(p.N, p.K);
    FewArgs f{};
    F8Args &a = f.a;
    a.w = {p.packed, p.packed + l.planes, l.rows};
    a.expert = l.bytes;
    a.scale_cols = l.cols;
    a.blocks = (int)l.blocks;
    a.M = p.rows;
    a.N = p.N;
    a.experts = p.experts;
    a.offsets = p.offsets;
    a.C = p.C;
    a.ldc = p.ldc;
    a.alpha = 1.0f;
    a.wide = can_store4(p.C, p.ldc, p.bf16 ? 2 : 4);
    f.K = p.K;
    if (p.K == 0) {
        const unsigned grid = (unsigned)(p.rows < 65536 ? p.rows : 65536);
        return p.bf16 ? launch(f8_zero_kernel<__bf16>, dim3(grid), dim3(256), 0, s, a)
                      : launch(f8_zero_kernel<float>, dim3(grid), dim3(256), 0, s, a);
    }
    const unsigned char *codes = nullptr;
    if (p.in == F8_IN_ROWS) {
        codes = (const unsigned char *)p.A;
    } else if (rows_first(p.rows, p.K, p.experts, p.offsets != nullptr)) {
        const hipError_t st =
            p.check ? hipSuccess
                    : launch_f8_rows({p.rows, p.K, p.A, p.lda, p.in, p.type, p.workspace}, s);
        if (st != hipSuccess) return st;
        codes = p.workspace;
    } else {
        f.A = p.A;
        f.lda = p.lda;
    }
    if (codes != nullptr) a.x = {codes, codes + f8_row_planes(p.rows, l.blocks), p.rows};
    if (p.type == F8_E4M3)
        return p.bf16 ? launch_product<F8_E4M3, __bf16>(p, f, s)
                      : launch_product<F8_E4M3, float>(p, f, s);
    return p.bf16 ? launch_product<F8_E5M2, __bf16>(p, f, s)
                  : launch_product<F8_E5M2, float>(p, f, s);
}

}  // namespace

// A call that its last launch refuses enqueues nothing: that is found out first.
hipError_t launch_f8(const F8Problem &given, hipStream_t s) {
    F8Problem p = given;
    if (p.K > 0) {
        p.check = true;
        const hipError_t st = run_f8(p, s);
        if (st != hipSuccess) return st;
    }
    p.check = false;
    return run_f8(p, s);
}

namespace {

int64_t ta_blocks(int rows, int experts, bool by_expert) {
    if (rows == 0) return 0;
    return by_expert ? most_blocks(rows, experts, kF8Block) : f8_blocks(rows);
}

int64_t whole16(__int128 bytes) { return (int64_t)((bytes + 15) / 16 * 16); }

template <class T, int WT, int XT>
hipError_t launch_ta_as(const F8TaProblem &p, const F8Args &a, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + T::BM - 1) / T::BM;
    const int64_t tiles_n = ((int64_t)p.N + T::BN - 1) / T::BN;
    const __int128 groups = (__int128)tiles_m * tiles_n * p.experts;
    if (groups > most_groups(T::THREADS)) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    return launch(f8_ta_kernel<T, WT, XT>, dim3((unsigned)groups), dim3(T::THREADS), 0, s, a, p.rows,
                  (int)tiles_m, (int)tiles_n);
}

}  // namespace

__int128 f8_ta_workspace(int rows, int M, int N, int experts) {
    if (rows == 0 || M == 0 || N == 0 || experts == 0) return 0;
    const int64_t blocks = ta_blocks(rows, experts, true);
    const __int128 a = f8_rows_bytes(M, blocks), d = f8_rows_bytes(N, blocks);
    return (a + 15) / 16 * 16 + (d + 15) / 16 * 16;
}

namespace {

hipError_t run_f8_ta(const F8TaProblem &p, hipStream_t s) {
    const bool product = p.rows > 0 && p.alpha != 0.0f;
    const int64_t blocks = product ? ta_blocks(p.rows, p.experts, true) : 0;
    F8Args a{};
    if (product && !p.check) {
        unsigned char *qa = p.workspace, *qd = qa + whole16(f8_rows_bytes(p.M, blocks));
        hipError_t st = launch_f8_columns(
            {p.rows, p.M, p.experts, p.offsets, p.A, p.lda, p.a_in, p.a_type, blocks, qa}, s);
        if (st != hipSuccess) return st;
        st = launch_f8_columns(
            {p.rows, p.N, p.experts, p.offsets, p.D, p.ldd, p.d_in, p.d_type, blocks, qd}, s);
        if (st != hipSuccess) return st;
        a.x = {qa, qa + f8_row_planes(p.M, blocks), p.M};
        a.w = {qd, qd + f8_row_planes(p.N, blocks), p.N};
    }
    a.blocks = (int)blocks;
    a.M = p.M;
    a.N = p.N;
    a.experts = p.experts;
    a.offsets = p.offsets;
    a.C = p.C;
    a.ldc = p.ldc;
    a.stridec = p.stridec;
    a.alpha = p.alpha;
    a.beta = p.beta;
    a.wide = can_store4(p.C, p.ldc, 4) && p.stridec % 4 == 0;
    if (p.d_type == F8_E4M3)
        return p.a_type == F8_E4M3 ? launch_ta_as<Tile128, F8_E4M3, F8_E4M3>(p, a, s)
                                   : launch_ta_as<Tile128, F8_E4M3, F8_E5M2>(p, a, s);
    return p.a_type == F8_E4M3 ? launch_ta_as<Tile128, F8_E5M2, F8_E4M3>(p, a, s)
                               : launch_ta_as<Tile128, F8_E5M2, F8_E5M2>(p, a, s);
}

}  // namespace

hipError_t launch_f8_ta(const F8TaProblem &given, hipStream_t s) {
    F8TaProblem p = given;
    p.check = true;
    const hipError_t st = run_f8_ta(p, s);
    p.check = false;
    return st != hipSuccess ? st : run_f8_ta(p, s);
}

}  // namespace sgemm
