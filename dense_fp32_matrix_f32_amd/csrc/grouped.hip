// grouped.hip -- the products of experts' rows, one launch for all experts: a
// work-group finds its expert from the device's offsets and computes one block of that
// expert's product, with the block kernel of mfma_kernel.h or, for a few rows of each
// expert, with one of its own.
#include "experts.h"
#include "groups.h"
#include "mfma_kernel.h"

namespace sgemm {

namespace {

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
constexpr int kFewRows = 16, kFewCols = 64;  // a block of grouped_few_kernel

// One block of C: rows from `first` on of expert e, whose rows end at `end`, and column
// block tn.
template <class C>
__device__ __forceinline__ void grouped_block(const GroupedProblem &p, float *lds, int e,
                                              int first, int end, int tn) {
    // the expert's matrices from this block's first row on
    const GemmArgs g{end - first, p.N, p.K, p.A + (int64_t)first * p.lda, p.lda,
                     p.B + e * p.strideb, p.ldb, p.C + (int64_t)first * p.ldc, p.ldc,
                     p.alpha, p.beta};
    const int n_lo = tn * C::BN;
    int m0 = 0, n0 = n_lo;
    edge_origin<C>(g.M, g.N, m0, n0);
    Acc<C> acc;
    zero_acc<C>(acc);
    mma_tile<C>(g, lds, m0, n0, 0, (g.K + C::BK - 1) / C::BK, acc);
    const int r_first = KwReduce<C>::run(lds, acc);
    store_tile<C>(g, m0, n0, acc, 0, n_lo, r_first, KwReduce<C>::RPG);
}

// Blocks of C.  Row blocks are counted expert by expert (find_block); the launch
// holds the most there can be, and the work-groups past those there are leave at
// once.  The ones there are get the XCD-aware order of the plain product, over all
// experts' row blocks: those of one expert follow each other and share its matrix.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC) void grouped_kernel(GroupedProblem p,
                                                                    int tiles_n) {
    __shared__ __attribute__((aligned(16))) float lds[C::LDS_FLOATS];
    // (offsets that are no running sum can give more blocks than were launched, or a
    // count that wrapped to a negative one)
    const int tiles_m = min(count_blocks(p.offsets, p.experts, p.rows, AllBlocks{C::BM}),
                            (int)(gridDim.x / (unsigned)tiles_n));
    if ((int)blockIdx.x >= tiles_m * tiles_n) return;
    int tm, tn, e, first, end;
    tile_order(blockIdx.x, tiles_m, tiles_n, C::GROUP_M, &tm, &tn);
    if (!find_block(p.offsets, p.experts, p.rows, C::BM, tm, &e, &first, &end)) return;
    grouped_block<C>(p, lds, e, first, end, tn);
}

// The same with blocks of two sizes: the experts' full blocks of L::BM rows, and after
// them (in the order of the launch, where they fill the CUs as the large ones end) the
// rows that are left, in blocks of S::BM.
template <class L, class S>
__global__ __launch_bounds__(L::THREADS, L::OCC) void grouped_mixed_kernel(GroupedProblem p,
                                                                          int large_n,
                                                                          int small_n) {
    static_assert(L::THREADS == S::THREADS && L::OCC == S::OCC, "one launch");
    constexpr int FLOATS = L::LDS_FLOATS > S::LDS_FLOATS ? L::LDS_FLOATS : S::LDS_FLOATS;
    __shared__ __attribute__((aligned(16))) float lds[FLOATS];
    const FullBlocks full{L::BM};
    const RestBlocks rest{L::BM, S::BM};
    const int large_m = max(0, min(count_blocks(p.offsets, p.experts, p.rows, full),
                                   (int)(gridDim.x / (unsigned)large_n)));
    int tm, tn, e, first, end, index, id = blockIdx.x;
    if (id < large_m * large_n) {
        tile_order(id, large_m, large_n, L::GROUP_M, &tm, &tn);
        if (!find_expert(p.offsets, p.experts, p.rows, full, tm, &e, &first, &end, &index)) return;
        first += index * L::BM;
        if (first >= 0 && first < end) grouped_block<L>(p, lds, e, first, end, tn);
        return;
    }
    id -= large_m * large_n;
    const int small_m = min(count_blocks(p.offsets, p.experts, p.rows, rest),
                            (int)(gridDim.x / (unsigned)small_n));
    if (id >= small_m * small_n) return;
    tile_order(id, small_m, small_n, S::GROUP_M, &tm, &tn);
    if (!find_expert(p.offsets, p.experts, p.rows, rest, tm, &e, &first, &end, &index)) return;
    first += (end - first) / L::BM * L::BM + index * S::BM;
    if (first >= 0 && first < end) grouped_block<S>(p, lds, e, first, end, tn);
}

// Few rows of each expert: bound by reading the matrices once.  A work-group forms up
// to 16 rows by 64 columns; its eight waves take units of 32 k in turn and their sums
// are added at the end, in a fixed order.  Operands go from memory to the 16x16x4
// matrix instruction without LDS: lane group q = lane / 16 holds k = 4q .. 4q+3 of
// each 16, so a 16-byte load is a row of A, or of a transposed B, for four
// instructions; of B as given it is four columns of one k, one for each of four
// instructions whose columns are 4i + e (i = lane % 16, e = the instruction).  B as given
// is loaded past the caches, a unit at a time (48 rows, 8 experts of 2048 x 4096: 45.7
// us, 5.9 TB/s; through the caches 51.9; two units in flight 48.6, three 54.6, with
// fewer waves).  B transposed is loaded by halves of a cache line and keeps its place
// in the caches, two units in flight (53.5 us; past the caches 62; one unit 57 to 72).
template <bool TB>
__global__ __launch_bounds__(512) void grouped_few_kernel(GroupedProblem p, int row_blocks) {
    constexpr int W = 8, COLS = kFewCols, UNIT = 32;
    __shared__ float red[W][kFewRows][COLS + 1];
    const int lane = threadIdx.x & 63, q = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // row blocks of one expert and strip follow each other: they share its B in one L2
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const int n0 = id / (unsigned)row_blocks * COLS;
    int expert, first, end;
    if (!find_block(p.offsets, p.experts, p.rows, kFewRows, id % (unsigned)row_blocks, &expert,
                    &first, &end))
        return;
    const int rows = min(kFewRows, end - first);
    const float *a = p.A + (int64_t)(first + min(i, rows - 1)) * p.lda + 4 * q;
    const float *mat = p.B + expert * p.strideb;
    // this lane's columns: n0 + 16u + i (B transposed), or four from `col` on, which at
    // the right edge are the last four
    const int col = TB ? 0 : min(n0 + 4 * i, p.N - 4);
    const float *b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        b[u] = TB ? mat + (int64_t)min(n0 + 16 * u + i, p.N - 1) * p.ldb + 4 * q
                  : mat + (int64_t)(4 * q + u) * p.ldb + col;

    struct Unit {
        f32x4 a[2], b[2][4];
    };
    auto load = [&](Unit &x, int unit) {
        const int64_t k = (int64_t)unit * UNIT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x.a[h] = load16(a + k + 16 * h);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float *from = b[u] + (TB ? k + 16 * h : (k + 16 * h) * p.ldb);
                x.b[h][u] = TB ? load16(from)
                               : __builtin_nontemporal_load((const f32x4_any *)from);
            }
        }
    };
    f32x4 acc[4] = {};
    auto multiply = [&](const Unit &x) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        x.a[h][j], TB ? x.b[h][e][j] : x.b[h][j][e], acc[e], 0, 0, 0);
    };

    // Units wave, wave + W, ..., the loads of the next D always issued before one is used
    // (past the last they repeat it).  With B transposed the rows of all strips would start
    // on the same memory channels, so strips start a pass of the waves apart.
    const int units = p.K / UNIT, n = (units - wave + W - 1) / W;
    if (n > 0) {
        constexpr int D = TB ? 2 : 1;
        const int rot = TB ? (int)(id / (unsigned)row_blocks * W % (unsigned)units) : 0;
        auto at = [&](int t) {
            const int unit = wave + min(t, n - 1) * W + rot;
            return unit >= units ? unit - units : unit;
        };
        Unit x[D];
#pragma unroll
        for (int u = 0; u < D; ++u) load(x[u], at(u));
        int t = 0;
        for (; t + D < n; t += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                multiply(x[u]);
                load(x[u], at(t + u + D));
            }
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (t + u < n) multiply(x[u]);
    }
    // the last k, fewer than a unit
    if (p.K % UNIT != 0 && wave == units % W) {
        const int k0 = units * UNIT;
        Unit x;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + 16 * h + j;  // and 4q more
                const bool in = k + 4 * q < p.K;
                x.a[h][j] = in ? a[k] : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (TB)
                        x.b[h][e][j] = in ? b[e][k] : 0.0f;
                    else
                        x.b[h][j][e] = in ? b[j][(int64_t)(k - j) * p.ldb + e] : 0.0f;
                }
            }
        multiply(x);
    }

#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int at = TB ? 16 * e + i : col + e - n0;
        if (!TB && at < 4 * i) continue;  // another lane's column
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][4 * q + r][at] = acc[e][r];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < rows * COLS; o += 64 * W) {
        const int m = o / COLS, c = o % COLS;
        if (n0 + c >= p.N) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[w][m][c];
        float *dst = p.C + (int64_t)(first + m) * p.ldc + n0 + c;
        *dst = epilogue(sum, p.alpha, p.beta, dst);
    }
}

// The expert whose rank by rows, most first, is `rank` (by number among equal ones): the
// shortest blocks then end a launch (8192 rows of 16 experts, 2048 x 2048, 540 -> 526 us,
// 4096 of 8, 1024 x 1024, 85 -> 82).  With more experts than 16 the expert of
// that number (8192 rows of 64, 1024 x 2048: 348 against 386).  Called by every lane of a
// wave.
__device__ __forceinline__ int expert_by_size(const int *__restrict__ offsets, int experts,
                                              int rows, int rank) {
    if (experts > 16) return rank;
    const int e = min((int)threadIdx.x & 63, experts - 1);
    const int lo = clamp_row(offsets[e], rows);
    const int mine = max(lo, clamp_row(offsets[e + 1], rows)) - lo;
    int before = 0;
    for (int other = 0; other < experts; ++other) {
        const int theirs = __builtin_amdgcn_readlane(mine, other);
        before += theirs > mine || (theirs == mine && other < e);
    }
    return __builtin_ctzll(__ballot(before == rank));
}

// Blocks of every C_e; the k loop of a block runs over its expert's rows.  Each
// expert's blocks are spread over all XCDs, so experts of different sizes load them
// alike.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC) void grouped_ta_kernel(GroupedTaProblem p,
                                                                       int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(16))) float lds[C::LDS_FLOATS];
    const int tiles = tiles_m * tiles_n;
    const int t = blockIdx.x % tiles;
    const int e = expert_by_size(p.offsets, p.experts, p.rows, blockIdx.x / tiles);
    const int lo = clamp_row(p.offsets[e], p.rows);
    const int hi = max(lo, clamp_row(p.offsets[e + 1], p.rows));
    const GemmArgs g{p.M, p.N, hi - lo, p.A + (int64_t)lo * p.lda, p.lda,
                     p.D + (int64_t)lo * p.ldd, p.ldd, p.C + e * p.stridec, p.ldc,
                     p.alpha, p.beta};
    int tm, tn;
    tile_order(t, tiles_m, tiles_n, C::GROUP_M, &tm, &tn);
    const int m_lo = tm * C::BM, n_lo = tn * C::BN;
    int m0 = m_lo, n0 = n_lo;
    edge_origin<C>(g.M, g.N, m0, n0);
    Acc<C> acc;
    zero_acc<C>(acc);
    int r_first = 0;
    if (g.K > 0 && p.alpha != 0.0f) {
        mma_tile<C>(g, lds, m0, n0, 0, (g.K + C::BK - 1) / C::BK, acc);
        r_first = KwReduce<C>::run(lds, acc);
    }
    store_tile<C>(g, m0, n0, acc, m_lo, n_lo, r_first, KwReduce<C>::RPG);
}

// C rows of experts = beta * C (no product: alpha == 0 or K == 0).
__global__ __launch_bounds__(256) void grouped_scale_kernel(GroupedProblem p) {
    for (int e = 0; e < p.experts; ++e) {
        const int lo = clamp_row(p.offsets[e], p.rows);
        const int hi = max(lo, clamp_row(p.offsets[e + 1], p.rows));
        for (int i = lo + blockIdx.x; i < hi; i += gridDim.x)
            for (int n = threadIdx.x; n < p.N; n += 256) {
                float *c = p.C + (int64_t)i * p.ldc + n;
                *c = p.beta == 0.0f ? 0.0f : p.beta * *c;
            }
    }
}

// Every offset inside a block's window fits 31 bits (as narrow_offsets()).
bool narrow(int64_t rows, int64_t ld, int64_t row_len) {
    return ((rows - 1) * ld + row_len) * 4 < ((int64_t)1 << 31);
}

template <class C>
hipError_t launch_blocks(const GroupedProblem &p, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + C::BN - 1) / C::BN;
    const int64_t blocks = most_blocks(p.rows, p.experts, C::BM) * tiles_n;
    if (blocks > most_groups(C::THREADS)) return hipErrorInvalidValue;
    return launch(grouped_kernel<C>, dim3((unsigned)blocks), dim3(C::THREADS), 0, s, p,
                  (int)tiles_n);
}

// Full blocks of T, the rest in blocks of U (with R register sets).
template <class T, class U, bool TB, int R>
hipError_t launch_mixed(const GroupedProblem &p, hipStream_t s) {
    if (!narrow(T::BM, p.lda, T::BK) ||
        !(TB ? narrow(T::BN, p.ldb, T::BK) : narrow(T::BK, p.ldb, T::BN)))
        return launch_blocks<Cfg<TileSmall, false, TB, false, 1>>(p, s);
    using L = Cfg<T, false, TB, true, 1>;
    using S = Cfg<U, false, TB, true, R>;
    const int64_t large_n = ((int64_t)p.N + L::BN - 1) / L::BN;
    const int64_t small_n = ((int64_t)p.N + S::BN - 1) / S::BN;
    const int64_t with_rows = p.rows < p.experts ? p.rows : p.experts;
    const int64_t rest = with_rows * (L::BM / S::BM);  // at most
    const int64_t blocks = p.rows / L::BM * large_n + rest * small_n;
    if (blocks > most_groups(L::THREADS)) return hipErrorInvalidValue;
    return launch(grouped_mixed_kernel<L, S>, dim3((unsigned)blocks), dim3(L::THREADS), 0, s, p,
                  (int)large_n, (int)small_n);
}

template <bool TB>
hipError_t launch_few(const GroupedProblem &p, hipStream_t s) {
    const int64_t row_blocks = most_blocks(p.rows, p.experts, kFewRows);
    const int64_t groups = ((int64_t)p.N + kFewCols - 1) / kFewCols * row_blocks;
    if (groups > most_groups(512)) return hipErrorInvalidValue;
    return launch(grouped_few_kernel<TB>, dim3((unsigned)groups), dim3(512), 0, s, p,
                  (int)row_blocks);
}

// Configuration T of the plain product with R register sets; rows so long that an
// offset inside a block passes 31 bits take 64-bit addresses (on one configuration).
template <class T, bool TB, int R>
hipError_t launch_grouped_tile(const GroupedProblem &p, hipStream_t s) {
    if (narrow(T::BM, p.lda, T::BK) &&
        (TB ? narrow(T::BN, p.ldb, T::BK) : narrow(T::BK, p.ldb, T::BN)))
        return launch_blocks<Cfg<T, false, TB, true, R>>(p, s);
    return launch_blocks<Cfg<TileSmall, false, TB, false, 1>>(p, s);
}

template <class C>
hipError_t launch_ta_blocks(const GroupedTaProblem &p, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + C::BM - 1) / C::BM;
    const int64_t tiles_n = ((int64_t)p.N + C::BN - 1) / C::BN;
    const __int128 blocks = (__int128)tiles_m * tiles_n * p.experts;
    if (blocks > most_groups(C::THREADS)) return hipErrorInvalidValue;
    return launch(grouped_ta_kernel<C>, dim3((unsigned)blocks), dim3(C::THREADS), 0, s, p,
                  (int)tiles_m, (int)tiles_n);
}

template <class T>
hipError_t launch_grouped_ta_tile(const GroupedTaProblem &p, hipStream_t s) {
    if (narrow(T::BK, p.lda, T::BM) && narrow(T::BK, p.ldd, T::BN))
        return launch_ta_blocks<Cfg<T, true, false, true, 1>>(p, s);
    return launch_ta_blocks<Cfg<TileSmall, true, false, false, 1>>(p, s);
}

// The configuration by the rows an expert has on average (the host knows no more).
// Smaller blocks waste less of the last block of each expert, larger ones read the
// operands less often.  Times in us, B as given / transposed, the experts uneven:
//   rows, experts, N x K      32x32        64x64     128x128   192x128   128x128, rest 64x64
//     48, 8, 4096 x 2048     55 / 68     73 / 78   129 / 231  193 / 362
//    512, 64, 1024 x 512     33 / 34     42 / 40    69 / 70    99 / 98
//    400, 8, 4096 x 2048     95 / 92    102 / 124  131 / 231  199 / 367
//    700, 8, 4096 x 2048    149 / 151   134 / 132  230 / 232  195 / 366    168 / 157
//    600, 2, 4096 x 4096                188 / 186                          271 / 273
//   3000, 4, 1000 x 1000                 69 /  69                           74 /  75
//   1500, 8, 4096 x 2048                244 / 236                          234 / 235
//   8192, 64, 2048 x 1024               383 / 375                          373 / 386
//   8192, 8, 4096 x 2048   1220 / 1192 1103 / 1096 1060 / 1146 1067 / 1071  996 / 1010
//  16384, 4, 4096 x 4096   4768 / 4769 4179 / 4300 3932 / 3945 3848 / 3888 3770 / 3787
//  30000, 4, 2048 x 2048                                       1779 / 1794 1783 / 1842
// (the first two rows against 54 and 27 us to read the matrices at 5 TB/s, the last three
// against 893, 3570 and 1634 us at the 154 TFLOP/s of a large plain product).  The blocks
// of two sizes are taken where there is almost one large one for every CU (0.93 to 1.0,
// measured at 0.85 and 0.98), or a second round over the CUs is nearly half full (last
// column: large blocks for a CU):
//   rows, experts, N x K        64x64      two sizes
//   3500,  8, 1024 x  512       42 /  40    44 /  45     0.85
//   4000,  8, 1024 x  512       50 /  50    44 /  45     0.98
//   7521, 17,  754 x 2376      260 / 273   295 / 275     1.38
//   3441,  9, 1795 x  910      113 / 122   113 / 115     1.57
//   2500,  8, 4096 x 2048      370 / 375   353 / 375     2.4
//   5400,  8, 4096 x 2048      745 / 744   700 / 708     5.3
// 32 x 32 blocks
// with B as given have one register set for few rows on many work-groups, two else; the
// kernel for few rows needs the many work-groups too, whether B is transposed or not:
//   rows, experts, N x K       few rows   one set / two / transposed
//     48,  8, 4096 x 2048       46 / 54    55 /  69 /  65
//     80,  8, 4096 x 2048       58 / 74    58 /  72 /  69
//    200,  8, 4096 x 2048       80 / 89     - /  71 /  67
//    512, 64, 1024 x  512       28 / 32    33 /  44 /  37
//    400, 64, 2048 x 1024       93 / 108    - / 126 / 122
//    256, 16, 2048 x 2048       62 / 74    60 /  75 /  68
//     48,  8, 2048 x 2048       32 / 45    44 /  32 /  34   (one work-group a CU)
//      4,  1, 4096 x 4096       29 / 35    43 /  27 /  26
template <bool TB>
hipError_t launch_grouped_as(const GroupedProblem &p, hipStream_t s) {
    const int each = p.rows / p.experts;
    // large blocks for a CU, if there were no rows past the full ones
    const double large = p.rows / 128.0 * std::ceil(p.N / 128.0) / compute_units();
    if (each > 128 && (large >= 1.45 || (large >= 0.93 && large <= 1.0)))
        return launch_mixed<TileWide, TileSmall, TB, 3>(p, s);
    if (each > 64) return launch_grouped_tile<TileSmall, TB, 3>(p, s);
    if (((int64_t)p.N + kFewCols - 1) / kFewCols * p.experts >= 2 * compute_units()) {
        if (each <= 8 && p.N >= 4) return launch_few<TB>(p, s);
        if constexpr (!TB) {
            if (each <= 16) return launch_grouped_tile<TileTiny, TB, 1>(p, s);
        }
    }
    return launch_grouped_tile<TileTiny, TB, 2>(p, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem &p, hipStream_t s) {
    if (p.K == 0 || p.alpha == 0.0f) {
        const unsigned grid = (unsigned)(p.rows < 65536 ? p.rows : 65536);
        return launch(grouped_scale_kernel, dim3(grid), dim3(256), 0, s, p);
    }
    return p.tb ? launch_grouped_as<true>(p, s) : launch_grouped_as<false>(p, s);
}

// 128 x 128 blocks where there are many for each CU, 64 x 64 else (8192 rows; the
// experts' numbers of rows differ, and so do the times of their blocks):
//   experts, M x N       64x64   128x128   large blocks a CU
//    4, 1100 x 1024     171-197  225-252     1.1
//    8, 1024 x 1024     137-139  136-154     2
//    8, 1024 x 1280     170-172  175-199     2.5
//    9,  910 x 1795     242-243  248-256     4.2
//    5, 2048 x 2048       517      470       5
//    8, 2048 x 4096      1020      980      16     (893 at the rate of a large product)
// and with 48 rows, 8, 2048 x 4096, 78 against 68 (54 to write the result at 5 TB/s).
hipError_t launch_grouped_ta(const GroupedTaProblem &p, hipStream_t s) {
    const double large = std::ceil(p.M / 128.0) * std::ceil(p.N / 128.0) * p.experts;
    return large > 4.5 * compute_units() ? launch_grouped_ta_tile<TileWide>(p, s)
                                   : launch_grouped_ta_tile<TileSmall>(p, s);
}

}  // namespace sgemm
