// grouped.hip -- the products of experts' rows, one launch for all experts, on
// the block kernel of mfma_kernel.h: a work-group finds its expert from the
// device's offsets and computes one block of that expert's product.
#include "experts.h"
#include "groups.h"
#include "mfma_kernel.h"

namespace sgemm {

namespace {

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
    const int tiles_m = min(count_blocks(p.offsets, p.experts, p.rows, C::BM),
                            (int)(gridDim.x / (unsigned)tiles_n));
    if ((int)blockIdx.x >= tiles_m * tiles_n) return;
    int tm, tn;
    tile_order(blockIdx.x, tiles_m, tiles_n, C::GROUP_M, &tm, &tn);
    int e, first, end;
    if (!find_block(p.offsets, p.experts, p.rows, C::BM, tm, &e, &first, &end)) return;
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

// Blocks of every C_e; the k loop of a block runs over its expert's rows.  Each
// expert's blocks are spread over all XCDs, so experts of different sizes load them
// alike.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC) void grouped_ta_kernel(GroupedTaProblem p,
                                                                       int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(16))) float lds[C::LDS_FLOATS];
    const int tiles = tiles_m * tiles_n;
    const int e = blockIdx.x / tiles, t = blockIdx.x % tiles;
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
//   rows, experts, N x K      32x32        64x64     128x128   192x128
//     48, 8, 4096 x 2048     55 / 68     73 / 78   129 / 231  193 / 362
//    512, 64, 1024 x 512     33 / 34     42 / 40    69 / 70    99 / 98
//    400, 8, 4096 x 2048     95 / 92    102 / 124  131 / 231  199 / 367
//    700, 8, 4096 x 2048    149 / 151   134 / 132  230 / 232  195 / 366
//   8192, 8, 4096 x 2048   1220 / 1192 1041 / 1069 1060 / 1146 1067 / 1071
//  16384, 4, 4096 x 4096   4768 / 4769 4179 / 4300 3932 / 3945 3848 / 3888
// (the first two rows against 54 and 27 us to read the matrices at 5 TB/s, the last two
// against 893 and 3570 us at the 154 TFLOP/s of a large plain product).  32 x 32 blocks
// with B as given: one register set is faster for the fewest rows (48 rows: 55 against
// 65, 512 rows 33 against 38), two for more (400 rows: 95 against 110).
template <bool TB>
hipError_t launch_grouped_as(const GroupedProblem &p, hipStream_t s) {
    const int each = p.rows / p.experts;
    if (each >= 4096) return launch_grouped_tile<TileTall, TB, 1>(p, s);
    if (each > 64) return launch_grouped_tile<TileSmall, TB, 3>(p, s);
    if constexpr (!TB) {
        if (each <= 16) return launch_grouped_tile<TileTiny, TB, 1>(p, s);
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

// 128 x 128 blocks unless they leave CUs without one (8192 rows, 8 experts, 2048 x
// 4096: 971 us against 1015 on 64 x 64 blocks, 893 at the rate of a large plain
// product; 48 rows: 68 against 78 us, 54 to write the result at 5 TB/s; 300 rows, 8
// experts, 512 x 512, 128 of the large blocks: 10.1 against 7.9).
hipError_t launch_grouped_ta(const GroupedTaProblem &p, hipStream_t s) {
    const double large = std::ceil(p.M / 128.0) * std::ceil(p.N / 128.0) * p.experts;
    return large > compute_units() ? launch_grouped_ta_tile<TileWide>(p, s)
                                   : launch_grouped_ta_tile<TileSmall>(p, s);
}

}  // namespace sgemm
