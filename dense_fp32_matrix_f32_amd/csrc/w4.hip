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
//     truncation of what is left, 8 bits at a time; only bits below 2^-133, bf16's
//     smallest number, are lost).  The parts of a row are rows of their own in the
//     matrix instruction: five rows of A fill one instruction of 16;
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
#include <type_traits>

#include "groups.h"
#include "w4.h"

namespace sgemm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

// The lane that cuts k = 4*(lane % 32) .. +3 of a block writes one half of a run: the
// run of lane part q of step j, 4*j + q, holds the eight k that w4_k(q, ..) names.
__device__ __forceinline__ int run_of(int lane) {
    const int k = 4 * (lane & 31);
    return k / 32 * 4 + w4_part(k % 32);
}
__device__ __forceinline__ int half_of(int lane) { return w4_index(4 * (lane & 31) % 32) / 4; }

// LDS holds, for each run of 8 k, 16-byte slots of the instruction rows.  Within each
// 16 rows a row's slot is permuted by the run's number: the writers of one row (two
// lanes a run) then fill all 64 banks once, and so do the lanes that a 16-byte read
// serves in one cycle (with a padded pitch instead, two fifths of the LDS cycles of
// the kernel for many rows were conflicts).
__device__ __forceinline__ int slot_of(int row, int run) { return row ^ run; }

// Writes by some lanes of a wave are read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// How a work-group's MR rows of A meet the matrix instructions of 16 rows.  A lane
// loads XV float4 vectors of A for a block of 128 k.
//   few rows: the three parts of row m are instruction rows 3m .. 3m+2, so 2 or 5
//   rows take one instruction and 10 take two; the parts' sums are added at the end.
//   A wave loads two rows at a time and hands the parts to the lanes that need them
//   through LDS;
//   16 rows:  each part is an instruction of its own and all three add into the
//   same registers, which leaves a third of the registers and of the scaling.  A lane
//   loads the values that it needs itself and cuts them in registers.
template <int XV_>
struct Rows {
    static constexpr int XV = XV_;
    static constexpr int MR = XV == 1 ? 2 : XV == 3 ? 5 : XV == 5 ? 10 : 16;
    static constexpr bool ADD = MR == 16;
    static constexpr int AT = (3 * MR + 15) / 16;  // operands of 16 rows
    static constexpr int RT = ADD ? 1 : AT;        // results of 16 rows
};

// Where a lane finds its share of a record.  The loads take no branch on the type
// of the scales or on whether there are zero points: the compiler then knows how
// many loads are in flight and waits for the block it needs, not for all of them.
// Two columns share PARTS words of 16-bit scales, of which a lane takes its half.
template <int PARTS>
struct Lane {
    unsigned code, scale, zero;  // byte offsets in a record
    bool f32, f16, odd, zeros;

    __device__ __forceinline__ Lane(const W4Layout &l, int lane) {
        const int col = lane & 15;
        f32 = l.scale_type == W4_F32;
        f16 = l.scale_type == W4_F16;
        odd = col & 1;
        zeros = l.zeros;
        code = 16 * lane;
        scale = kW4Codes + (f32 ? 4 * PARTS * col : 2 * PARTS * (col & ~1));
        zero = zeros ? kW4Codes + PARTS * kW4Cols * l.scale_size + PARTS * col : 0;
    }
};

// The lane's codes, scales and zero points of a block.
template <int PARTS>
struct Record {
    uint4 codes;
    unsigned scale[PARTS];
    unsigned zero;

    __device__ __forceinline__ void load(const unsigned char *rec, const Lane<PARTS> &at) {
        codes = *(const uint4 *)(rec + at.code);
        __builtin_memcpy(scale, __builtin_assume_aligned(rec + at.scale, 4 * PARTS), 4 * PARTS);
        const unsigned char *z = rec + at.zero;
        zero = PARTS == 1 ? *z : PARTS == 2 ? *(const unsigned short *)z : *(const unsigned *)z;
    }
    __device__ __forceinline__ float scale_of(int t, const Lane<PARTS> &at) const {
        unsigned half;
        if constexpr (PARTS == 1) {
            half = at.odd ? scale[0] >> 16 : scale[0] & 0xFFFFu;
        } else {
            const unsigned w = at.odd ? scale[PARTS / 2 + t / 2] : scale[t / 2];
            half = t % 2 ? w >> 16 : w & 0xFFFFu;
        }
        const float wide = (float)__builtin_bit_cast(_Float16, (unsigned short)half);
        const float narrow = __builtin_bit_cast(float, half << 16);
        return at.f32 ? __builtin_bit_cast(float, scale[t]) : at.f16 ? wide : narrow;
    }
    __device__ __forceinline__ float zero_of(int t, const Lane<PARTS> &at) const {
        return at.zeros ? (float)((zero >> (8 * t)) & 255) : 8.0f;
    }
    __device__ __forceinline__ unsigned word(int j) const {
        return j == 0 ? codes.x : j == 1 ? codes.y : j == 2 ? codes.z : codes.w;
    }
};

// Four values of a row of A from k on, K >= 4: in the last ones of a row, those that
// end at K, which last_k() then puts in their places with zeros past K.
__device__ __forceinline__ f32x4 load_k(const float *row, int k, int K) {
    f32x4 x;
    __builtin_memcpy(&x, row + min(k, K - 4), 16);
    return x;
}

__device__ __forceinline__ f32x4 last_k(f32x4 x, int k, int K) {
    const int by = k - min(k, K - 4);  // places to move down; 4 and more: all past K
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v = 0.0f;
#pragma unroll
        for (int f = e; f < 4; ++f)
            if (by == f - e) v = x[f];
        y[e] = v;
    }
    return y;
}

// Four values of A as three parts, 8 bytes each.
__device__ __forceinline__ void store_parts(f32x4 x, unsigned char *p0, unsigned char *p1,
                                            unsigned char *p2) {
    const f32x4 y = {lower(x[0]), lower(x[1]), lower(x[2]), lower(x[3])};
    const f32x4 z = {lower(y[0]), lower(y[1]), lower(y[2]), lower(y[3])};
    *(uint2 *)p0 = uint2{upper(x[0], x[1]), upper(x[2], x[3])};
    *(uint2 *)p1 = uint2{upper(y[0], y[1]), upper(y[2], y[3])};
    *(uint2 *)p2 = uint2{upper(z[0], z[1]), upper(z[2], z[3])};
}

// Eight values of a row of A as the operands of its three parts.
__device__ __forceinline__ void cut_parts(f32x4 lo, f32x4 hi, bf16x8 (&a)[3]) {
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        const Frag f{.word = {upper(lo[0], lo[1]), upper(lo[2], lo[3]), upper(hi[0], hi[1]),
                              upper(hi[2], hi[3])}};
        a[part] = f.v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = lower(lo[e]);
            hi[e] = lower(hi[e]);
        }
    }
}

// The value of the lane whose number differs in bit D (1, 2 or 4).
template <int D>
__device__ __forceinline__ float lane_xor(float x) {
    if constexpr (D == 4) {
        // within 8 lanes: the mirror image, which after the steps of 1 and 2 holds the
        // same sum as the lane 4 away
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                             0, __builtin_bit_cast(int, x), 0x141, 0xf, 0xf, true));
    } else {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x),
                                               D == 1 ? 0xB1 : 0x4E, 0xf, 0xf, true));
    }
}

// R rows, CT strips of columns, PARTS scales of a column in a block, the loads of D
// blocks in flight in each wave.
constexpr int W = 8;  // waves

template <class R, int CT, int PARTS, int D>
__global__ __launch_bounds__(W * 64) void w4_kernel(W4Layout l, W4Problem p, int row_blocks) {
    constexpr int MR = R::MR, RT = R::RT, AT = R::AT, XV = R::XV;
    constexpr int RP = 16 * AT;       // 16-byte slots of one run of 8 k in LDS
    constexpr int STEPS = 4 / PARTS;  // matrix instructions of 32 k under one scale
    constexpr int COLS = kW4Cols * CT;
    constexpr int XS = R::ADD ? 0 : 16 * RP * 16;  // bytes of a wave's parts of A
    constexpr int RED = 16 * RT * (COLS + 1) * 4;  // bytes of a wave's sums
    __shared__ __attribute__((aligned(16))) unsigned char lds[W * (XS > RED ? XS : RED)];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // row blocks of one strip follow each other: they share its weights in one L2
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const unsigned row_block = id % (unsigned)row_blocks;
    const int strip0 = id / (unsigned)row_blocks * CT;
    int expert = 0, first = row_block * MR, end = p.rows;
    if (p.offsets != nullptr &&
        !find_block(p.offsets, p.experts, p.rows, MR, row_block, &expert, &first, &end))
        return;
    const int rows = min(MR, end - first);

    const unsigned char *strip[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        strip[c] = p.packed + expert * l.expert_bytes +
                   min(strip0 + c, l.strips - 1) * l.strip_bytes;
    // vector i of this lane: four k from k_of(i) of a block on, of row arow[i]
    constexpr int AROWS = R::ADD ? 1 : XV;
    const float *arow[AROWS];
#pragma unroll
    for (int i = 0; i < AROWS; ++i)
        arow[i] = p.A + (int64_t)(first + min(R::ADD ? lane & 15 : 2 * i + (lane >> 5), rows - 1)) *
                            p.lda;
    auto k_of = [&](int i) {
        return R::ADD ? 32 * (i / 2) + w4_k(lane >> 4, 4 * (i % 2)) : 4 * (lane & 31);
    };

    // One block of 128 k in registers.
    struct Block {
        Record<PARTS> w[CT];
        f32x4 x[XV];
    };
    const Lane<PARTS> at(l, lane);
    auto load = [&](Block &b, int block) {
#pragma unroll
        for (int c = 0; c < CT; ++c) b.w[c].load(strip[c] + (int64_t)block * l.record, at);
#pragma unroll
        for (int i = 0; i < XV; ++i)
            b.x[i] = load_k(arow[R::ADD ? 0 : i], block * kW4Block + k_of(i), l.K);
    };

    // in LDS: this lane's four k of row 2i + lane/32, and its operand of step j
    unsigned char *xs = lds + wave * XS;
    const int put_run = run_of(lane);
    unsigned char *put = xs + put_run * RP * 16 + half_of(lane) * 8;
    auto put_at = [&](int row) { return put + slot_of(row, put_run) * 16; };
    auto get = [&](int j, int r) {
        const int run = 4 * j + (lane >> 4);
        return *(const bf16x8 *)(xs + (run * RP + slot_of(lane & 15, run) + 16 * r) * 16);
    };

    f32x4 total[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) total[r][c] = f32x4{};

    const Frag ones{.word = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};

    auto process = [&](Block &b, int block) {
        if (block * kW4Block + kW4Block > l.K) {
#pragma unroll
            for (int i = 0; i < XV; ++i)
                b.x[i] = last_k(b.x[i], block * kW4Block + k_of(i), l.K);
        }
        if constexpr (!R::ADD) {
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                if (2 * i + 1 >= MR && (lane >> 5)) continue;
                const int row = 3 * (2 * i + (lane >> 5));
                store_parts(b.x[i], put_at(row), put_at(row + 1), put_at(row + 2));
            }
            wave_sync();
        }
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
            // column c < CT; sums of A in column CT
            f32x4 sum[RT][CT + 1];
#pragma unroll
            for (int u = 0; u < STEPS; ++u) {
                const int j = t * STEPS + u;
                bf16x8 a[AT], q[CT + 1];
                if constexpr (R::ADD) {
                    cut_parts(b.x[2 * j], b.x[2 * j + 1], a);
                } else {
#pragma unroll
                    for (int r = 0; r < AT; ++r) a[r] = get(j, r);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) q[c] = codes_of(b.w[c].word(j));
                q[CT] = ones.v;
#pragma unroll
                for (int r = AT - 1; r >= 0; --r)
#pragma unroll
                    for (int c = 0; c <= CT; ++c) {
                        f32x4 &out = sum[R::ADD ? 0 : r][c];
                        const bool start = u == 0 && (!R::ADD || r == AT - 1);
                        out = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            a[r], q[c], start ? f32x4{} : out, 0, 0, 0);
                    }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float s = b.w[c].scale_of(t, at), z = b.w[c].zero_of(t, at);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[r][c][e] =
                            fmaf(s, fmaf(-z, sum[r][CT][e], sum[r][c][e]), total[r][c][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!R::ADD) wave_sync();
    };

    // Blocks wave, wave + W, ...: the loads of the next D are always issued before
    // one is used; past the last block they repeat it.
    const int n = (l.blocks - wave + W - 1) / W;
    if (n > 0) {
        Block b[D];
#pragma unroll
        for (int u = 0; u < D; ++u) load(b[u], wave + min(u, n - 1) * W);
        int i = 0;
        for (; i + D < n; i += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                process(b[u], wave + (i + u) * W);
                load(b[u], wave + min(i + u + D, n - 1) * W);
            }
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (i + u < n) process(b[u], wave + (i + u) * W);
    }

    // Add the waves' sums (and the parts' rows), smallest part first, then by wave.
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
    for (int o = threadIdx.x; o < rows * COLS; o += W * 64) {
        const int m = o / COLS, col = o % COLS, n_at = strip0 * kW4Cols + col;
        if (n_at >= l.N) continue;
        float sum = 0.0f;
#pragma unroll
        for (int part = R::ADD ? 0 : 2; part >= 0; --part)
#pragma unroll
            for (int w = 0; w < W; ++w)
                sum += red[(w * 16 * RT + (R::ADD ? m : 3 * m + part)) * (COLS + 1) + col];
        p.C[(int64_t)(first + m) * p.ldc + n_at] = sum;
    }
}

template <class R, int CT, int D>
hipError_t launch_rows(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    const int64_t row_blocks = p.offsets != nullptr ? most_blocks(p.rows, p.experts, R::MR)
                                                    : ((int64_t)p.rows + R::MR - 1) / R::MR;
    const int64_t groups = ((int64_t)l.strips + CT - 1) / CT * row_blocks;
    if (groups > most_groups(W * 64)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)groups), block(W * 64);
    switch (l.parts) {
    case 4: return launch(w4_kernel<R, CT, 4, D>, grid, block, 0, s, l, p, (int)row_blocks);
    case 2: return launch(w4_kernel<R, CT, 2, D>, grid, block, 0, s, l, p, (int)row_blocks);
    default: return launch(w4_kernel<R, CT, 1, D>, grid, block, 0, s, l, p, (int)row_blocks);
    }
}

// ---------------------------------------------------------------------------
// Many rows.  Cutting A into parts costs about six vector operations a value, and
// in the kernel above every work-group cuts its rows for 16 to 64 columns only.
// Here a work-group computes 16 or 32 rows by 128 to 512 columns over all k, its waves
// side by side in columns, and A is cut once for all of them, into two stages of LDS:
// while one block of 128 k is multiplied, the next one's x is cut, one barrier a block.
// The sums of A over 32 k (for the zero points) are formed on the way, in fp32.
template <int W_, int RTW_, int CTW_, int D_>
struct Wide {
    static constexpr int D = D_;  // blocks of 128 k whose loads are in flight (even)
    static constexpr int RTW = RTW_, CTW = CTW_;  // 16-row and 16-column tiles of a wave
    static constexpr int BM = 16 * RTW, STRIPS = W_ * CTW, THREADS = 64 * W_;
    static constexpr int RP = 3 * BM;  // 16-byte slots of one run of 8 k in LDS
    static constexpr int XV = BM * 32 / THREADS;  // float4 vectors of A a lane and step
    static_assert(BM * 32 % THREADS == 0, "whole vectors");
};

template <class T, int PARTS>
__global__ __launch_bounds__(T::THREADS) void w4_wide_kernel(W4Layout l, W4Problem p,
                                                            int row_blocks) {
    constexpr int BM = T::BM, RP = T::RP, XV = T::XV, RTW = T::RTW, CTW = T::CTW;
    constexpr int STEPS = 4 / PARTS;
    __shared__ __attribute__((aligned(16))) unsigned char xs[2][16 * RP * 16];
    __shared__ __attribute__((aligned(16))) float sums[2][4][BM];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // row blocks that read the same weights follow each other
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const unsigned row_block = id % (unsigned)row_blocks;
    const int strip0 = id / (unsigned)row_blocks * T::STRIPS + wave * CTW;
    int expert = 0, first = row_block * BM, end = p.rows;
    if (p.offsets != nullptr &&
        !find_block(p.offsets, p.experts, p.rows, BM, row_block, &expert, &first, &end))
        return;
    const int rows = min(BM, end - first);

    const unsigned char *strip[CTW];
#pragma unroll
    for (int c = 0; c < CTW; ++c)
        strip[c] = p.packed + expert * l.expert_bytes +
                   min(strip0 + c, l.strips - 1) * l.strip_bytes;
    // vector v of this work-item: four k of row (tid + v * THREADS) / 32
    constexpr int VROWS = T::THREADS / 32;
    const int k_lane = 4 * (tid & 31);
    const float *a0 = p.A + (int64_t)first * p.lda;
    unsigned arow[XV];  // element offsets of the vectors' rows (wide_fits())
#pragma unroll
    for (int v = 0; v < XV; ++v)
        arow[v] = (unsigned)min(tid / 32 + v * VROWS, rows - 1) * (unsigned)p.lda;

    struct Block {
        Record<PARTS> w[CTW];
    };
    const Lane<PARTS> at(l, lane);
    auto load_w = [&](Block &b, int block) {
#pragma unroll
        for (int c = 0; c < CTW; ++c) b.w[c].load(strip[c] + (int64_t)block * l.record, at);
    };
    auto load_x = [&](f32x4(&x)[XV], int block) {
        const unsigned k = min(block * kW4Block + k_lane, l.K - 4);
#pragma unroll
        for (int v = 0; v < XV; ++v) __builtin_memcpy(&x[v], a0 + (arow[v] + k), 16);
    };
    auto last_x = [&](f32x4(&x)[XV], int block) {
        if (block * kW4Block + kW4Block > l.K) {
#pragma unroll
            for (int v = 0; v < XV; ++v) x[v] = last_k(x[v], block * kW4Block + k_lane, l.K);
        }
    };
    auto cut = [&](f32x4 x, int v, int stage) {
        const int run = run_of(tid), row = tid / 32 + v * VROWS;
        unsigned char *to = xs[stage] + (run * RP + slot_of(row, run)) * 16 + half_of(tid) * 8;
        store_parts(x, to, to + BM * 16, to + 2 * BM * 16);
        // eight lanes hold 32 k of a row
        float t = (x[0] + x[1]) + (x[2] + x[3]);
        t += lane_xor<1>(t);
        t += lane_xor<2>(t);
        t += lane_xor<4>(t);
        if ((tid & 7) == 0) sums[stage][(tid & 31) >> 3][tid / 32 + v * VROWS] = t;
    };

    f32x4 total[RTW][CTW];
#pragma unroll
    for (int r = 0; r < RTW; ++r)
#pragma unroll
        for (int c = 0; c < CTW; ++c) total[r][c] = f32x4{};

    // The products of one block, in LDS stage `stage`, and between them the cutting of
    // the next block's x into the other stage.
    auto multiply = [&](const Block &b, const f32x4(&x)[XV], int stage) {
        auto get = [&](int j, int row) {
            const int run = 4 * j + (lane >> 4);
            return *(const bf16x8 *)(xs[stage] +
                                     (run * RP + slot_of(lane & 15, run) + row) * 16);
        };
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
            f32x4 sum[RTW][CTW];
#pragma unroll
            for (int u = 0; u < STEPS; ++u) {
                const int j = t * STEPS + u;
                bf16x8 a[RTW][3], q[CTW];
#pragma unroll
                for (int r = 0; r < RTW; ++r)
#pragma unroll
                    for (int part = 2; part >= 0; --part)
                        a[r][part] = get(j, part * BM + 16 * r);
#pragma unroll
                for (int c = 0; c < CTW; ++c) q[c] = codes_of(b.w[c].word(j));
                // a wave in its matrix instructions goes first, so that the other waves of
                // its SIMD unpack and cut in their shadow
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int c = 0; c < CTW; ++c)
#pragma unroll
                        for (int r = 0; r < RTW; ++r)
                            sum[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                a[r][part], q[c], u == 0 && part == 2 ? f32x4{} : sum[r][c], 0, 0,
                                0);
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int v = j * XV / 4; v < (j + 1) * XV / 4; ++v) cut(x[v], v, 1 - stage);
            }
            f32x4 sum_x[RTW];
#pragma unroll
            for (int r = 0; r < RTW; ++r) {
                const int at_row = 16 * r + 4 * (lane >> 4);
                sum_x[r] = *(const f32x4 *)&sums[stage][t * STEPS][at_row];
#pragma unroll
                for (int u = 1; u < STEPS; ++u)
                    sum_x[r] += *(const f32x4 *)&sums[stage][t * STEPS + u][at_row];
            }
#pragma unroll
            for (int c = 0; c < CTW; ++c) {
                const float s = b.w[c].scale_of(t, at), z = b.w[c].zero_of(t, at);
#pragma unroll
                for (int r = 0; r < RTW; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[r][c][e] =
                            fmaf(s, fmaf(-z, sum_x[r][e], sum[r][c][e]), total[r][c][e]);
            }
        }
    };

    // Register slots: w[i % D] holds block i, and x[i % D] until it is cut, a block
    // before its product.  Freed slots are loaded at once with the block D later (x
    // first: it is needed first); past the last block the loads repeat it.
    constexpr int D = T::D;
    static_assert(D % 2 == 0, "the LDS stage of a slot is a constant");
    f32x4 x[D][XV];
    Block w[D];
    auto clip = [&](int block) { return min(block, l.blocks - 1); };
#pragma unroll
    for (int i = 0; i < D; ++i) {
        load_x(x[i], clip(i));
        load_w(w[i], clip(i));
    }
    last_x(x[0], 0);
#pragma unroll
    for (int v = 0; v < XV; ++v) cut(x[0][v], v, 0);
    load_x(x[0], clip(D));
    __syncthreads();
    for (int block = 0; block < l.blocks; block += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (block + i < l.blocks) {
                last_x(x[(i + 1) % D], clip(block + i + 1));
                multiply(w[i], x[(i + 1) % D], i & 1);
            }
            load_x(x[(i + 1) % D], clip(block + i + 1 + D));
            load_w(w[i], clip(block + i + D));
            __syncthreads();
        }
    }

    // a lane holds rows 4 * (lane / 16) + e of each tile
#pragma unroll
    for (int r = 0; r < RTW; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = 16 * r + 4 * (lane >> 4) + e;
#pragma unroll
            for (int c = 0; c < CTW; ++c) {
                const int n = (strip0 + c) * kW4Cols + (lane & 15);
                if (m < rows && n < l.N) p.C[(int64_t)(first + m) * p.ldc + n] = total[r][c][e];
            }
        }
}

// Fewer than four k: no 16-byte vector of A lies inside a row.  One work-item for
// each element of C.
__global__ __launch_bounds__(256) void w4_short_kernel(W4Layout l, W4Problem p) {
    const int n = blockIdx.x * 256 + threadIdx.x, col = n % kW4Cols;
    for (int64_t i = blockIdx.y; i < p.rows; i += gridDim.y) {
        int e = 0, row = (int)i, end;
        if (p.offsets != nullptr &&
            !find_block(p.offsets, p.experts, p.rows, 1, (int)i, &e, &row, &end))
            return;
        if (n >= l.N) continue;
        float sum = 0.0f;
        if (l.K > 0) {
            const unsigned char *rec = p.packed + e * l.expert_bytes + n / kW4Cols * l.strip_bytes;
            const unsigned word = *(const unsigned *)(rec + 16 * col);
            const int part = col * l.parts;  // the first part: k < 32
            const float s = w4_scale(rec + kW4Codes + part * l.scale_size, l.scale_type);
            const int z = l.zeros ? rec[kW4Codes + l.parts * kW4Cols * l.scale_size + part] : 8;
            for (int k = 0; k < l.K; ++k)
                sum = fmaf(p.A[row * p.lda + k],
                           (float)((int)(word >> w4_shift(w4_index(k)) & 15) - z), sum);
            sum *= s;
        }
        p.C[row * p.ldc + n] = sum;
    }
}

template <class T>
int64_t wide_blocks(const W4Problem &p) {
    return p.offsets != nullptr ? most_blocks(p.rows, p.experts, T::BM)
                                : ((int64_t)p.rows + T::BM - 1) / T::BM;
}

// Work-groups of the kernel for many rows.
template <class T>
int64_t wide_groups(const W4Layout &l, const W4Problem &p) {
    return ((int64_t)l.strips + T::STRIPS - 1) / T::STRIPS * wide_blocks<T>(p);
}

// Every offset of a row block's rows fits 32 bits.
template <class T>
bool wide_fits(const W4Layout &l, const W4Problem &p) {
    return (T::BM - 1) * p.lda + l.K < ((int64_t)1 << 32);
}

template <class T, int PARTS>
hipError_t launch_wide(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    const int64_t groups = wide_groups<T>(l, p);
    if (groups > most_groups(T::THREADS)) return hipErrorInvalidValue;
    return launch(w4_wide_kernel<T, PARTS>, dim3((unsigned)groups), dim3(T::THREADS), 0, s, l, p,
                  (int)wide_blocks<T>(p));
}

// 16 rows by 128 or 256 columns, or 32 by 512 (32 by 256 with four scales of a column
// in a block, which need more registers than the larger leaves).  A larger block cuts A
// for more columns and unpacks codes for more rows, but fewer of them fill the CUs less
// evenly and waste more of an expert's last one.  So the largest is taken where its
// rounds over the CUs are at least four fifths full (for experts, from 512 rows each on),
// and of the others 16 by 256 where it nearly fills the CUs and is not just past that.
// With four scales 16 by 256 gains nothing over 16 by 128.  Times in us:
//                                          16 x 128  16 x 256  largest
//   128 rows 4096 x 4096, group 64           26        37
//   256 rows 4096 x 4096, group 128          36        33        85
//   320 rows 4096 x 4096, group 64           51        56        93
//   700 rows 4096 x 4096, group 128          96        80        86
//   512 rows 8192 x 4096, group 128         133       109        88
//   1024 rows 4096 x 4096, group 64         141       119        95
//   512 rows by expert, 16 x 2048 x 2048     28        31
//   1000 rows by expert, 64 x 2048 x 1024    30        26        50
//   2048 rows by expert, 8 x 4096 x 2048    145       121       134
//   4096 rows by expert, 8 x 4096 x 2048    283       237       224
//   300 rows 4096 x 4096, group 32           62        79        64
//   512 rows 4096 x 4096, group 32           82        81        65
//   700 rows 4096 x 4096, group 32          117       119       126
//   256 by expert, 16 x 1408 x 4096, 32      42        41        64
//   2000 by expert, 16 x 1408 x 4096, 32    124       160       128
using Wide128 = Wide<8, 1, 1, 2>;
using Wide256 = Wide<8, 1, 2, 2>;

template <int PARTS>
hipError_t launch_wide_as(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    using Largest = typename std::conditional<PARTS == 4, Wide<8, 2, 2, 2>, Wide<8, 2, 4, 2>>::type;
    const int64_t cus = compute_units();
    const int64_t largest = wide_groups<Largest>(l, p), rounds = (largest + cus - 1) / cus;
    if (5 * largest >= 4 * cus * rounds && (p.offsets == nullptr || p.rows / p.experts >= 512))
        return launch_wide<Largest, PARTS>(l, p, s);
    if constexpr (PARTS < 4) {
        const int64_t groups = wide_groups<Wide256>(l, p);
        if (groups >= cus * 5 / 8 && (groups <= cus || groups > cus * 3 / 2))
            return launch_wide<Wide256, PARTS>(l, p, s);
    }
    return launch_wide<Wide128, PARTS>(l, p, s);
}

// Whether there are rows enough for these kernels, and their offsets fit.
bool many_rows(const W4Layout &l, const W4Problem &p) {
    return wide_groups<Wide128>(l, p) >= compute_units() && wide_fits<Wide<8, 2, 4, 2>>(l, p);
}

hipError_t launch_many_rows(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    switch (l.parts) {
    case 4: return launch_wide_as<4>(l, p, s);
    case 2: return launch_wide_as<2>(l, p, s);
    default: return launch_wide_as<1>(l, p, s);
    }
}

}  // namespace

// The kernel for a call, by the rows that share a reading of the weights (for
// experts, if each had the same number) and the strips.  Times in us, back to back,
// random data, the weights of three calls in turn (8.7 MB for 4096 x 4096):
//   rows  N x K, group      choice           others
//   1     4096 x 4096, 128  one strip 4.5    two 5.3; 4 waves 5.3, 16 waves 4.6
//   1     8192 x 8192, 128  one strip 9.5    two 9.4; 4 waves 10.2, 16 waves 9.5
//   8 by expert, 64 x 2048 x 2048, 128: two strips 6.8, one 8.1 (1024 work-groups; between
//                           512 and that neither was measured)
//   5     4096 x 4096, 64   5-row form 5.5   10-row form 6.9
//   8     4096 x 4096, 128  10-row form 6.8  16-row form 7.9
//   16    4096 x 4096, 128  one strip 9.7    two 10.2, four 13.0; 10-row form 9.7
//   16    8192 x 8192, 64   two strips 19.1  one 32.8, four 24.6
//   16    5120 to 7168 x 8192, 64  one strip 33 (12 rows 28): more work-groups than CUs, but
//                           not the 512 from which two strips are taken; two not measured
//   32    4096 x 4096, 128  two strips 10.6  one 17.2, four 13.5
//   256 by expert, 16 x 1408 x 4096, 32: many rows 42, two strips 44, one 64, four 49
//   256 by expert, 16 x 2048 x 2048, 128: many rows 19, two strips 26
//   64    4096 x 4096, 128  four strips 14.1 two 18.9; many rows 32
//   128   4096 x 4096, 64   many rows 25.6   four strips 27.0, two 35.2
//   128   8192 x 4096, 128  many rows 33.2   four strips 32.9
//   256   4096 x 4096, 128  many rows 33     four strips 49
//   512   4096 x 4096, 32   many rows 65     four strips 121
//   512   8192 x 4096, 128  many rows 88     four strips 197
// (4.5 us is 1.9 TB/s; a kernel that does nothing takes about 2.5.)  Slices of k over
// several work-groups, their sums added by a second kernel, brought 16 x 8192 x 8192
// from 17.9 to 17.0 us and were not kept.
hipError_t launch_w4(const W4Layout &l, const W4Problem &p, hipStream_t s) {
    if (l.K < 4) {
        const dim3 grid((unsigned)((l.N + 255ll) / 256),
                        (unsigned)(p.rows < 65535 ? p.rows : 65535));
        return launch(w4_short_kernel, grid, dim3(256), 0, s, l, p);
    }
    const int experts = p.offsets != nullptr ? p.experts : 1;
    const int64_t each = ((int64_t)p.rows + experts - 1) / experts;
    if (each <= 2) {
        const int64_t row_blocks = p.offsets != nullptr ? most_blocks(p.rows, experts, 2) : 1;
        const int64_t groups = l.strips * row_blocks;
        return groups >= 1024 ? launch_rows<Rows<1>, 2, 2>(l, p, s)
                              : launch_rows<Rows<1>, 1, 2>(l, p, s);
    }
    if (each <= 5) return launch_rows<Rows<3>, 1, 1>(l, p, s);
    if (each <= 10) return launch_rows<Rows<5>, 1, 1>(l, p, s);
    if (many_rows(l, p)) return launch_many_rows(l, p, s);
    const int64_t groups = l.strips * ((each + 15) / 16 * experts);
    if (groups >= 1024 && l.parts < 4) return launch_rows<Rows<8>, 4, 1>(l, p, s);
    if (groups >= 512) return launch_rows<Rows<8>, 2, 1>(l, p, s);
    return launch_rows<Rows<8>, 1, 1>(l, p, s);
}

}  // namespace sgemm
