// grouped.hip -- the products of experts' rows, one launch for all experts, on
// the block kernel of mfma_kernel.h: a work-group finds its expert from the
// device's offsets and computes one block of that expert's product.
#include "experts.h"
#include "groups.h"
#include "mfma_kernel.h"

namespace sgemm {

namespace {

// Blocks of C: row blocks are counted expert by expert (find_block), so the launch
// holds the most there can be and the rest of the work-groups leave at once.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC) void grouped_kernel(GroupedProblem p, int tiles_n) {
    __shared__ __attribute__((aligned(16))) float lds[C::LDS_FLOATS];
    const int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
    int e, first, end;
    if (!find_block(p.offsets, p.experts, p.rows, C::BM, tm, &e, &first, &end)) return;
    // the expert's matrices from this block's first row on
    const GemmArgs g{end - first, p.N, p.K, p.A + (int64_t)first * p.lda, p.lda,
                     p.B + e * p.strideb, p.ldb, p.C + (int64_t)first * p.ldc, p.ldc,
                     p.alpha, p.beta};
    const int m_lo = 0, n_lo = tn * C::BN;
    int m0 = m_lo, n0 = n_lo;
    edge_origin<C>(g.M, g.N, m0, n0);
    Acc<C> acc;
    zero_acc<C>(acc);
    mma_tile<C>(g, lds, m0, n0, 0, (g.K + C::BK - 1) / C::BK, acc);
    const int r_first = KwReduce<C>::run(lds, acc);
    store_tile<C>(g, m0, n0, acc, m_lo, n_lo, r_first, KwReduce<C>::RPG);
}

// Blocks of every C_e; the k loop of a block runs over its expert's rows.
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
    const int m_lo = t / tiles_n * C::BM, n_lo = t % tiles_n * C::BN;
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

using Tile = MfmaTile<64, 64, 16, 32, 32, 1, 4, 3>;

// Every offset inside a block's window fits 31 bits (as narrow_offsets()).
bool narrow(int64_t rows, int64_t ld, int64_t row_len) {
    return ((rows - 1) * ld + row_len) * 4 < ((int64_t)1 << 31);
}

template <class T, bool TB>
hipError_t launch_grouped_tile(const GroupedProblem &p, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + T::BN - 1) / T::BN;
    const int64_t blocks = most_blocks(p.rows, p.experts, T::BM) * tiles_n;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(T::THREADS);
    const bool nar = narrow(T::BM, p.lda, T::BK) &&
                     (TB ? narrow(T::BN, p.ldb, T::BK) : narrow(T::BK, p.ldb, T::BN));
    if (nar)
        return launch(grouped_kernel<Cfg<T, false, TB, true, 1>>, grid, block, 0, s, p,
                      (int)tiles_n);
    return launch(grouped_kernel<Cfg<T, false, TB, false, 1>>, grid, block, 0, s, p, (int)tiles_n);
}

template <class T>
hipError_t launch_grouped_ta_tile(const GroupedTaProblem &p, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + T::BM - 1) / T::BM;
    const int64_t tiles_n = ((int64_t)p.N + T::BN - 1) / T::BN;
    const __int128 blocks = (__int128)tiles_m * tiles_n * p.experts;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(T::THREADS);
    const bool nar = narrow(T::BK, p.lda, T::BM) && narrow(T::BK, p.ldd, T::BN);
    if (nar)
        return launch(grouped_ta_kernel<Cfg<T, true, false, true, 1>>, grid, block, 0, s, p,
                      (int)tiles_m, (int)tiles_n);
    return launch(grouped_ta_kernel<Cfg<T, true, false, false, 1>>, grid, block, 0, s, p,
                  (int)tiles_m, (int)tiles_n);
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem &p, hipStream_t s) {
    if (p.K == 0 || p.alpha == 0.0f) {
        const unsigned grid = (unsigned)(p.rows < 65536 ? p.rows : 65536);
        return launch(grouped_scale_kernel, dim3(grid), dim3(256), 0, s, p);
    }
    return p.tb ? launch_grouped_tile<Tile, true>(p, s) : launch_grouped_tile<Tile, false>(p, s);
}

hipError_t launch_grouped_ta(const GroupedTaProblem &p, hipStream_t s) {
    return launch_grouped_ta_tile<Tile>(p, s);
}

}  // namespace sgemm
