// layer.hip -- a whole layer of experts for a few tokens, in two kernels.
//
//     h[t][j] = act(x[t] G_e) * (x[t] U_e)   or act(x[t] U_e),   e = ids[t][j]
//     y[t]    = sum over j of w[t][j] * h[t][j] D_e
//
// With few tokens the layer is bound by reading the matrices of the experts that were
// chosen, once each.  Both kernels work on items: up to MR pairs (token, choice) of one expert,
// MR being the rows that a matrix instruction holds.  In the first a work-group takes one item and a
// strip of columns of both G and U, whose products meet in its epilogue.  In the second it
// takes a strip of D's columns and all items in turn, or a share of their blocks of k, and adds
// what they give, with its weight, to the tokens' sums in LDS, each wave to its own.  Where several
// work-groups share a strip, as they do where there are few strips for the CUs, each writes
// its sums to the workspace and a third kernel adds those.  The waves take blocks of k in turn,
// and whatever is added is added in a fixed order.
//
// Up to 64 pairs the kernels find the items themselves; more are sorted by expert first
// (route.hip), which is a launch more.  More than kLayerTokens tokens go in several rounds.
#include <initializer_list>
#include <type_traits>

#include "experts.h"
#include "groups.h"
#include "layer.h"
#include "parts.h"

namespace sgemm {

namespace {

// ---- weights in 4 and 8 bits: strips of 16 columns, blocks of 128 k ----------------------------

// Where a lane finds its share of a strip, and in which order of k it is: eight k of
// step j (of four) are run read_run(j, g) of LDS, g = lane / 16; the lane that holds k =
// 4 * (lane % 32) .. +3 of a row writes half put_half() of run put_run(); and vector i of a
// lane that holds its own k is k_of(i, g) .. +3.
template <int PARTS_>
struct FourBits {
    static constexpr int PARTS = PARTS_;
    static constexpr bool SUMS = true;  // zero points: the sums of the rows count too
    typedef Record<PARTS> Weights;
    W4Layout l;
    Lane<PARTS> at;
    __device__ FourBits(const LayerMatrices &m, int lane) : l(m.w4), at(m.w4, lane) {}
    __device__ const unsigned char *strip(const void *data, int expert, int s) const {
        return (const unsigned char *)data + expert * l.expert_bytes +
               min(s, l.strips - 1) * l.strip_bytes;
    }
    __device__ void load(Weights &w, const unsigned char *strip, int, int block) const {
        w.load(strip + (int64_t)block * l.record, at);
    }
    __device__ void arrived(Weights &) const {}
    __device__ bf16x8 operand(const Weights &w, int j) const { return codes_of(w.word(j)); }
    __device__ float scale(const Weights &w, int t) const { return w.scale_of(t, at); }
    __device__ float zero(const Weights &w, int t) const { return w.zero_of(t, at); }
    static __device__ int put_run(int lane) { return run_of(lane); }
    static __device__ int put_half(int lane) { return half_of(lane); }
    static __device__ int read_run(int j, int g) { return 4 * j + g; }
    static __device__ int k_of(int i, int g) { return 32 * (i / 2) + w4_k(g, 4 * (i % 2)); }
};

struct EightBits {
    static constexpr int PARTS = 1;
    static constexpr bool SUMS = false;
    struct Weights {
        uint4 c[2];
        float s;
    };
    F8Weights l;
    int code, flip;
    __device__ EightBits(const LayerMatrices &m, int lane) : l(m.f8) {
        const int i = lane & 15, place = f8_place(lane >> 4, i);
        code = i * kF8Block + place;
        flip = place & 64 ? -64 : 64;
    }
    __device__ const unsigned char *strip(const void *data, int expert, int s) const {
        return (const unsigned char *)data + expert * l.bytes +
               min((int64_t)s * 16, l.rows - 16) * kF8Block;
    }
    // s: the strip's number, for its scales; those of all strips lie after the planes
    __device__ void load(Weights &w, const unsigned char *strip, int s, int block) const {
        const int64_t n = min((int64_t)s * 16, l.rows - 16);
        const unsigned char *from = strip + block * l.rows * kF8Block + code;
        w.c[0] = *(const uint4 *)from;
        w.c[1] = *(const uint4 *)(from + flip);
        w.s = ((const float *)(strip - n * kF8Block + l.planes))[block * l.cols + n / kF8Block];
    }
    __device__ void arrived(Weights &w) const { w.s = f8_here(w.s); }
    __device__ bf16x8 operand(const Weights &w, int j) const {
        const uint4 c = w.c[j / 2];
        const unsigned lo = j % 2 ? c.z : c.x, hi = j % 2 ? c.w : c.y;
        const float power = f8_split(w.s).power;
        Frag f;
        f.pair[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, false);
        f.pair[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, true);
        f.pair[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, false);
        f.pair[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, true);
        return f.v;
    }
    __device__ float scale(const Weights &w, int) const { return f8_split(w.s).rest; }
    __device__ float zero(const Weights &, int) const { return 0.0f; }
    static __device__ int put_run(int lane) { return (lane & 31) >> 1; }
    static __device__ int put_half(int lane) { return lane & 1; }
    static __device__ int read_run(int j, int g) { return j < 2 ? 2 * g + j : 6 + 2 * g + j; }
    static __device__ int k_of(int i, int g) { return 64 * (i / 4) + 16 * g + 4 * (i % 4); }
};

// Engines: the products of up to MR rows with NW matrices, 16 CT / NW columns of each, a block of
// BLOCK k at a time.  A lane's results are total[RT][CT] of four rows each: tile c, element e
// of tile row r is row result_row(r, e) (several parts of a row add up to it) and column
// column(c).

// Weights in 4 and 8 bits; rows in one of the forms of parts.h.
template <class R, class F, int NW, int STRIPS>
struct CodesEngine {
    static constexpr int MR = R::MR, RT = R::RT, CT = NW * STRIPS, COLS = 16 * STRIPS;
    static constexpr int BLOCK = kW4Block;
    static constexpr int XV = R::XV, AT = R::AT, RP = 16 * AT;
    static constexpr int AROWS = R::ADD ? 1 : XV;
    static constexpr int XS = R::ADD ? 0 : 16 * RP * 16;  // bytes of a wave's parts in LDS
    static constexpr int STEPS = 4 / F::PARTS;
    // Sums kept apart.  The matrix instruction cuts what it adds at the last bits of its largest term,
    // and with a zero point the sum is larger than what is left of it: the two smaller parts of 16
    // rows then get sums of their own (without them the error of a layer of 2048 x 1024 in its
    // 2-norm is 2.2e-6 instead of 2.4e-7, and the calls of 16 tokens take 1 us less of 80).
    static constexpr int SETS = R::ADD && F::SUMS ? 2 : RT;

    struct Block {
        typename F::Weights w[CT];
        f32x4 x[XV];
    };
    F f;
    int lane;

    __device__ CodesEngine(const LayerMatrices &like, int lane_) : f(like, lane_), lane(lane_) {}

    // results: tile rows in the order in which their parts are to be added, smallest first
    __device__ int result_row(int r, int e) const {
        const int at = 16 * r + 4 * (lane >> 4) + e;
        return R::ADD ? at : at / 3;
    }
    __device__ int column(int c) const { return 16 * (c % STRIPS) + (lane & 15); }

    // row(m): row m of the item, m < MR
    template <class Row>
    __device__ __forceinline__ void load(Block &b, const LayerMatrices *const (&m)[NW], int expert,
                                         int n0, int block, int K, const Row &row) const {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int s = n0 / 16 + c % STRIPS;
            f.load(b.w[c], f.strip(m[c / STRIPS]->data, expert, s), s, block);
        }
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            const int k = R::ADD ? F::k_of(i, lane >> 4) : 4 * (lane & 31);
            const float *from = row(R::ADD ? lane & 15 : min(2 * i + (lane >> 5), MR - 1));
            b.x[i] = load_k(from, block * BLOCK + k, K);
        }
    }

    __device__ __forceinline__ void multiply(f32x4 (&total)[RT][CT], Block &b, int block, int K,
                                             unsigned char *xs) const {
        const int g = lane >> 4;
        if (block * BLOCK + BLOCK > K) {
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                const int k = R::ADD ? F::k_of(i, g) : 4 * (lane & 31);
                b.x[i] = last_k(b.x[i], block * BLOCK + k, K);
            }
        }
        if constexpr (!R::ADD) {
            const int run = F::put_run(lane);
            unsigned char *put = xs + run * RP * 16 + F::put_half(lane) * 8;
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                const int row = 3 * (2 * i + (lane >> 5));
                if (2 * i + 1 >= MR && (lane >> 5)) continue;
                store_parts(b.x[i], put + slot_of(row, run) * 16, put + slot_of(row + 1, run) * 16,
                            put + slot_of(row + 2, run) * 16);
            }
            wave_sync();
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) f.arrived(b.w[c]);
        const Frag ones{.word = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
        constexpr int CS = CT + (F::SUMS ? 1 : 0);
#pragma unroll
        for (int t = 0; t < F::PARTS; ++t) {
            f32x4 sum[SETS][CS];
#pragma unroll
            for (int u = 0; u < STEPS; ++u) {
                const int j = t * STEPS + u;
                bf16x8 a[AT], q[CS];
                if constexpr (R::ADD) {
                    cut_parts(b.x[2 * j], b.x[2 * j + 1], a);
                } else {
                    const int run = F::read_run(j, g);
#pragma unroll
                    for (int r = 0; r < AT; ++r)
                        a[r] = *(const bf16x8 *)(xs + (run * RP + slot_of(lane & 15, run) + 16 * r) * 16);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) q[c] = f.operand(b.w[c], j);
                if constexpr (F::SUMS) q[CT] = ones.v;
#pragma unroll
                for (int r = AT - 1; r >= 0; --r)
#pragma unroll
                    for (int c = 0; c < CS; ++c) {
                        const int set = !R::ADD ? r : SETS == 2 && r > 0;
                        f32x4 &out = sum[set][c];
                        const bool start =
                            u == 0 && (!R::ADD || r == AT - 1 || (SETS == 2 && r == 0));
                        out = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            a[r], q[c], start ? f32x4{} : out, 0, 0, 0);
                    }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float s = f.scale(b.w[c], t), z = f.zero(b.w[c], t);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = sum[r][c][e];
                        if constexpr (F::SUMS) v = fmaf(-z, sum[r][CS - 1][e], v);
                        if constexpr (F::SUMS && R::ADD)
                            v += fmaf(-z, sum[1][CS - 1][e], sum[1][c][e]);
                        total[r][c][e] = fmaf(s, v, total[r][c][e]);
                    }
            }
            // the next scales' operands wait: with them a lane would need more than 256 registers
            // (scales of 64 k, 16 tokens, 2 of 8 of 4096 x 4096: the first kernel 66 us, so 57)
            if constexpr (R::ADD && F::PARTS > 1) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!R::ADD) wave_sync();
    }
};

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// fp32 matrices (TB: given as N x K): 16 rows by 64 columns, 32 k at a time, operands straight
// from memory to the 16x16x4 matrix instruction as in grouped_few_kernel: lane group q =
// lane / 16 holds k = 4q .. 4q+3 of each 16; of a matrix as given four columns of one k, of a
// transposed one four k of a column.  At the edges the last k and columns are loaded
// again, without a branch, and then put aside.
template <bool TB, int NW>
struct PlainEngine {
    static constexpr int MR = 16, RT = 1, CT = 4 * NW, COLS = 64, BLOCK = 32, XS = 0;
    struct Block {
        f32x4 a[2], b[NW][2][4];
        int shift;  // columns that a lane's vectors lie left of their place
    };
    int lane;

    __device__ PlainEngine(const LayerMatrices &, int lane_) : lane(lane_) {}
    __device__ int result_row(int, int e) const { return 4 * (lane >> 4) + e; }
    __device__ int column(int c) const {
        const int t = c % 4, i = lane & 15;
        return TB ? 16 * t + i : 4 * i + t;
    }

    template <class Row>
    __device__ __forceinline__ void load(Block &x, const LayerMatrices *const (&m)[NW], int expert,
                                         int n0, int block, int K, const Row &row) const {
        const int q = lane >> 4, i = lane & 15, k0 = block * BLOCK, N = m[0]->columns;
        const float *from = row(i);
        x.shift = TB ? 0 : max(0, n0 + 4 * i - (N - 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + 16 * h + 4 * q;
            x.a[h] = load_k(from, k, K);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float *mat = (const float *)m[w]->data + expert * m[w]->stride;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if constexpr (TB)
                        x.b[w][h][u] = load_k(mat + min(n0 + 16 * u + i, N - 1) * m[w]->ld, k, K);
                    else
                        x.b[w][h][u] = __builtin_nontemporal_load(
                            (const f32x4_any *)(mat + min(k + u, K - 1) * m[w]->ld +
                                                min(n0 + 4 * i, N - 4)));
                }
            }
        }
    }

    __device__ __forceinline__ void multiply(f32x4 (&total)[RT][CT], Block &x, int block, int K,
                                             unsigned char *) const {
        if (block * BLOCK + BLOCK > K) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = block * BLOCK + 16 * h + 4 * (lane >> 4);
                x.a[h] = last_k(x.a[h], k, K);
#pragma unroll
                for (int w = 0; w < NW; ++w)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        x.b[w][h][u] = TB          ? last_k(x.b[w][h][u], k, K)
                                       : k + u < K ? x.b[w][h][u]
                                                   : f32x4{};
            }
        }
        if (!TB && __any(x.shift)) {  // past the last column anything may stand
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const f32x4 v = x.b[w][h][u];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int d = 1; e + d < 4; ++d)
                                if (x.shift == d) x.b[w][h][u][e] = v[e + d];
                    }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[0][4 * w + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            x.a[h][j], TB ? x.b[w][h][e][j] : x.b[w][h][j][e], total[0][4 * w + e],
                            0, 0, 0);
    }
};

// ---- activations --------------------------------------------------------------------------------

__device__ __forceinline__ float activate(float z, int act) {
    if (act == ACT_SILU) return z / (1.0f + expf(-z));
    if (act == ACT_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
    return z < 0.0f ? 0.0f : z;
}

// ---- items ----------------------------------------------------------------------------------------

struct Hidden {
    float *h;
    int64_t ld;
    const int *offsets, *order;  // of the sort, or NULL
    float *parts;                // of y, where work-groups share a strip's items
};

// Up to 64 pairs, a lane each: its expert (-1: none) and how many pairs before it have the same.  A
// pair that a multiple of MR others come before begins an item.
struct LanePair {
    int id, rank;
    __device__ explicit LanePair(const LayerProblem &p) {
        const int n = p.tokens * p.top, lane = threadIdx.x & 63;
        id = lane < n ? p.ids[lane / p.top * p.ldids + lane % p.top] : -1;
        if (id >= p.experts) id = -1;
        rank = 0;
        for (int q = 0; q < n; ++q)
            rank += __builtin_amdgcn_readlane(id, q) == id && q < lane;
    }
    template <int MR>
    __device__ bool begins() const {
        return id >= 0 && rank % MR == 0;
    }
};

__device__ __forceinline__ int bits_below(unsigned long long mask) {
    return __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
}

struct Item {
    int expert, rows;
};

// Item number `item`: its expert, its number of rows and its pairs (into LDS, for all waves).
template <int MR>
__device__ __forceinline__ bool find_item(const LayerProblem &p, const Hidden &o, int item,
                                          int *pairs, Item *out) {
    if (o.offsets != nullptr) {
        const int n = p.tokens * p.top;
        int first, end;
        if (!find_block(o.offsets, p.experts, n, MR, item, &out->expert, &first, &end)) return false;
        out->rows = min(MR, end - first);
        if ((int)threadIdx.x < out->rows)
            pairs[threadIdx.x] = max(0, min(o.order[first + threadIdx.x], n - 1));
    } else {
        const LanePair mine(p);
        const bool begins = mine.begins<MR>();
        const unsigned long long at =
            __ballot(begins && bits_below(__ballot(begins)) == item);
        if (at == 0) return false;
        const int lead = __builtin_ctzll(at);
        out->expert = __builtin_amdgcn_readlane(mine.id, lead);
        const int r0 = __builtin_amdgcn_readlane(mine.rank, lead);
        const bool member = mine.id == out->expert && mine.rank >= r0 && mine.rank < r0 + MR;
        out->rows = __popcll(__ballot(member));
        if (threadIdx.x < 64 && member) pairs[mine.rank - r0] = threadIdx.x;
    }
    __syncthreads();
    return true;
}

// All items, in LDS: item i has rows[i] pairs of expert[i], the pairs from first[i] on.  A token that
// has an expert twice counts once, with both weights (its two h are the same): `weight` of the
// first such pair is their sum and token[] of the others is -1.
struct Items {
    int *expert, *first, *rows, *pair, *token;
    float *weight;
};

template <int MR>
__device__ __forceinline__ int find_items(const LayerProblem &p, const Hidden &o, int most,
                                          const Items &s) {
    const int n = p.tokens * p.top, tid = threadIdx.x;
    int items;
    if (o.offsets != nullptr) {
        // every wave counts the items, the first one lists them
        items = 0;
        for (int base = 0; base < p.experts; base += 64) {
            const int e = base + (tid & 63);
            int lo = 0, hi = 0;
            if (e < p.experts) {
                lo = clamp_row(o.offsets[e], n);
                hi = max(lo, clamp_row(o.offsets[e + 1], n));
            }
            const int mine = (hi - lo + MR - 1) / MR, upto = wave_scan(mine);
            if (tid < 64) {
                for (int b = 0; b < mine; ++b) {
                    const int item = items + upto - mine + b;
                    if ((unsigned)item >= (unsigned)most) break;
                    s.expert[item] = e;
                    s.first[item] = lo + b * MR;
                    s.rows[item] = min(MR, hi - lo - b * MR);
                }
            }
            items += __builtin_amdgcn_readlane(upto, 63);
        }
        items = max(0, min(items, most));
        const int kept = clamp_row(o.offsets[p.experts], n);
        for (int q = tid; q < n; q += blockDim.x) {
            const int pair = q < kept ? max(0, min(o.order[q], n - 1)) : -1;
            s.pair[q] = pair;
            s.token[q] = pair < 0 ? -1 : pair / p.top;
            s.weight[q] = pair < 0 ? 0.0f : p.weights[pair / p.top * p.ldw + pair % p.top];
        }
        __syncthreads();
        // Pairs of one expert and token lie side by side: the first takes the others' weights.  (Pair
        // by pair, and the items from one walk over the experts: the second kernel for 64
        // tokens, 4 of 16, 8 bits, takes 37 us; item by item it took 44.)
        auto expert_of = [&](int pair) { return p.ids[pair / p.top * p.ldids + pair % p.top]; };
        for (int q = tid; q < kept; q += blockDim.x) {
            const int pair = s.pair[q], token = pair / p.top;
            auto same = [&](int other) {
                return other / p.top == token && expert_of(other) == expert_of(pair);
            };
            if (q > 0 && same(s.pair[q - 1])) {
                s.token[q] = -1;
            } else if (q + 1 < kept && same(s.pair[q + 1])) {
                float w = s.weight[q];
                for (int r = q + 1; r < kept && same(s.pair[r]); ++r)
                    w += p.weights[token * p.ldw + s.pair[r] % p.top];
                s.weight[q] = w;
            }
        }
    } else {
        const LanePair mine(p);
        const bool begins = mine.begins<MR>();
        const unsigned long long mask = __ballot(begins);
        items = __popcll(mask);
        if (tid < 64) {
            const int token = tid < n ? tid / p.top : -1;
            const float w = tid < n ? p.weights[token * p.ldw + tid % p.top] : 0.0f;
            int item = bits_below(mask), rows = 0;  // of a pair that begins one
            bool later = false;
            float sum = 0.0f;
            for (int q = 0; q < n; ++q) {
                const int id = __builtin_amdgcn_readlane(mine.id, q);
                const int rank = __builtin_amdgcn_readlane(mine.rank, q);
                const int other = __builtin_amdgcn_readlane(token, q);
                const float v = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), q));
                const bool same = id == mine.id;
                // the pair that begins this one's item comes before it
                const int its = __builtin_popcountll(mask & ((1ull << q) - 1));
                if (same && rank == mine.rank / MR * MR) item = its;
                rows += same && rank >= mine.rank && rank < mine.rank + MR;
                later |= same && other == token && q < tid;
                sum += same && other == token ? v : 0.0f;
            }
            if (mine.id >= 0) {
                const int at = item * MR + mine.rank % MR;
                s.pair[at] = tid;
                s.token[at] = later ? -1 : token;
                s.weight[at] = sum;
                if (begins) {
                    s.expert[item] = mine.id;
                    s.first[item] = item * MR;
                    s.rows[item] = rows;
                }
            }
        }
    }
    __syncthreads();
    return items;
}

// ---- first kernel: h ------------------------------------------------------------------------------

template <class E, bool GATED, int W, int D>
__global__ __launch_bounds__(W * 64, 2) void layer_up_kernel(LayerProblem p, Hidden o, int items) {
    constexpr int NW = GATED ? 2 : 1, PITCH = NW * E::COLS + 1, RED = 16 * E::RT * PITCH * 4;
    __shared__ __attribute__((aligned(16))) unsigned char lds[W * (E::XS > RED ? E::XS : RED)];
    __shared__ int pairs[E::MR];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // items of one strip follow each other
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const int n0 = id / (unsigned)items * E::COLS, K = p.width;
    Item mine;
    if (!find_item<E::MR>(p, o, id % (unsigned)items, pairs, &mine)) return;

    const E engine(p.up, lane);
    const LayerMatrices *m[NW];
    m[NW - 1] = &p.up;
    if constexpr (GATED) m[0] = &p.gate;
    auto load = [&](typename E::Block &b, int block) {
        engine.load(b, m, mine.expert, n0, block, K, [&](int r) {
            return p.x + pairs[min(r, mine.rows - 1)] / p.top * p.ldx;
        });
    };
    f32x4 total[E::RT][E::CT];
#pragma unroll
    for (int r = 0; r < E::RT; ++r)
#pragma unroll
        for (int c = 0; c < E::CT; ++c) total[r][c] = f32x4{};
    unsigned char *xs = lds + wave * E::XS;
    // Blocks wave, wave + W, ...: the loads of the next D are always issued before one is used;
    // past the last block they repeat it.
    const int blocks = (K + E::BLOCK - 1) / E::BLOCK, n = (blocks - wave + W - 1) / W;
    if (n > 0) {
        typename E::Block b[D];
#pragma unroll
        for (int u = 0; u < D; ++u) load(b[u], wave + min(u, n - 1) * W);
        int i = 0;
        for (; i + D < n; i += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                engine.multiply(total, b[u], wave + (i + u) * W, K, xs);
                load(b[u], wave + min(i + u + D, n - 1) * W);
            }
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (i + u < n) engine.multiply(total, b[u], wave + (i + u) * W, K, xs);
    }
    __syncthreads();
    float *red = (float *)lds;
#pragma unroll
    for (int r = 0; r < E::RT; ++r)
#pragma unroll
        for (int c = 0; c < E::CT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[wave * (RED / 4) + (16 * r + 4 * (lane >> 4) + e) * PITCH +
                    c / (E::CT / NW) * E::COLS + engine.column(c)] = total[r][c][e];
    __syncthreads();
    // instruction rows of a row: all of it, or three parts, of which the smallest goes first
    constexpr int PARTS = E::MR == 16 ? 1 : 3;
    auto sum_of = [&](int m, int col) {
        float sum = 0.0f;
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
            for (int w = 0; w < W; ++w)
                sum += red[w * (RED / 4) + (PARTS * m + part) * PITCH + col];
        return sum;
    };
    for (int q = threadIdx.x; q < mine.rows * E::COLS; q += W * 64) {
        const int m = q / E::COLS, col = q % E::COLS, at = n0 + col;
        if (at >= p.hidden) continue;
        float v = activate(sum_of(m, col), p.act);
        if constexpr (GATED) v *= sum_of(m, E::COLS + col);
        o.h[pairs[m] * o.ld + at] = v;
    }
}

// ---- second kernel: y -----------------------------------------------------------------------------

// In LDS: the waves' parts of the rows, their sums for all tokens, and the items.
template <class E, int W>
struct DownLds {
    int tokens, items, list;  // list: places in the pairs' arrays
    __host__ __device__ constexpr int sums() const { return W * E::XS; }
    __host__ __device__ constexpr int items_at() const {
        return sums() + W * tokens * (E::COLS + 1) * 4;
    }
    __host__ __device__ constexpr int bytes() const {
        return items_at() + 3 * items * 4 + 3 * list * 4;
    }
};

template <class E, int W, int D>
__global__ __launch_bounds__(W * 64) void layer_down_kernel(LayerProblem p, Hidden o, int most,
                                                            int list, int split) {
    extern __shared__ __attribute__((aligned(16))) unsigned char down_lds[];
    constexpr int PITCH = E::COLS + 1;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned id = xcd_remap(blockIdx.x, gridDim.x);
    const int n0 = id / (unsigned)split * E::COLS, share = id % (unsigned)split, K = p.hidden;
    const DownLds<E, W> at{p.tokens, most, list};
    float *sums = (float *)(down_lds + at.sums());
    int *table = (int *)(down_lds + at.items_at());
    const Items s{table, table + most, table + 2 * most, table + 3 * most, table + 3 * most + list,
                  (float *)(table + 3 * most + 2 * list)};
    for (int q = threadIdx.x; q < W * p.tokens * PITCH; q += W * 64) sums[q] = 0.0f;
    const int items = __builtin_amdgcn_readfirstlane(find_items<E::MR>(p, o, most, s));
    sums += wave * p.tokens * PITCH;

    const E engine(p.down, lane);
    const LayerMatrices *const m[1] = {&p.down};
    const int blocks = (K + E::BLOCK - 1) / E::BLOCK;
    // Unit u: block u % blocks of item u / blocks.  A work-group takes its share of them, a wave
    // every W-th.
    struct Unit {
        int item, block;
        int64_t left;  // units of the share from this one on
        __device__ void step(int by, int blocks) {
            left -= by;
            block += by;
            while (block >= blocks) {
                block -= blocks;
                ++item;
            }
        }
    };
    auto load = [&](typename E::Block &b, const Unit &u) {
        const int first = s.first[u.item], rows = s.rows[u.item];
        engine.load(b, m, __builtin_amdgcn_readfirstlane(s.expert[u.item]), n0, u.block, K,
                    [&](int r) { return o.h + s.pair[first + min(r, rows - 1)] * o.ld; });
    };
    f32x4 total[E::RT][E::CT];
    auto clear = [&] {
#pragma unroll
        for (int r = 0; r < E::RT; ++r)
#pragma unroll
            for (int c = 0; c < E::CT; ++c) total[r][c] = f32x4{};
    };
    // The item's sums, with their weights, to its tokens.  Lanes that add at once hold rows of
    // different tokens.
    auto flush = [&](int item) {
        const int first = s.first[item], rows = s.rows[item];
#pragma unroll
        for (int r = E::RT - 1; r >= 0; --r)
#pragma unroll
            for (int e = 3; e >= 0; --e) {
                const int row = engine.result_row(r, e);
                const int token = row < rows ? s.token[first + row] : -1;
                if (token < 0) continue;
                const float w = s.weight[first + row];
#pragma unroll
                for (int c = 0; c < E::CT; ++c) {
                    float *to = sums + token * PITCH + engine.column(c);
                    *to = fmaf(w, total[r][c][e], *to);
                }
            }
    };
    unsigned char *xs = down_lds + wave * E::XS;
    const int64_t units = (int64_t)items * blocks, lo = units * share / split;
    Unit now{(int)(lo / blocks), (int)(lo % blocks), units * (share + 1) / split - lo};
    now.step(wave, blocks);
    if (now.left > 0) {
        Unit next = now;
        typename E::Block b[D];
#pragma unroll
        for (int u = 0; u < D; ++u) {
            load(b[u], next);
            if (next.left > W) next.step(W, blocks);  // past the last unit it is loaded again
        }
        int item = now.item;
        clear();
        while (now.left > 0) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                if (now.left > 0) {
                    if (now.item != item) {
                        flush(item);
                        clear();
                        item = now.item;
                    }
                    engine.multiply(total, b[u], now.block, K, xs);
                }
                now.step(W, blocks);
                load(b[u], next);
                if (next.left > W) next.step(W, blocks);
            }
        }
        flush(item);
    }
    __syncthreads();
    sums = (float *)(down_lds + at.sums());
    for (int q = threadIdx.x; q < p.tokens * E::COLS; q += W * 64) {
        const int t = q / E::COLS, col = q % E::COLS;
        if (n0 + col >= p.width) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += sums[(w * p.tokens + t) * PITCH + col];
        if (split == 1)
            p.y[t * p.ldy + n0 + col] = sum;
        else
            o.parts[((int64_t)share * p.tokens + t) * p.width + n0 + col] = sum;
    }
}

// y from the shares' parts.
__global__ __launch_bounds__(256) void layer_join_kernel(LayerProblem p, Hidden o, int split) {
    const int64_t n = (int64_t)p.tokens * p.width;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float sum = 0.0f;
#pragma unroll 4
        for (int s = 0; s < split; ++s) sum += o.parts[s * n + i];
        p.y[i / p.width * p.ldy + i % p.width] = sum;
    }
}

// ---- fewer than four k, or nothing to add -------------------------------------------------------------

// One number of a matrix.
__device__ __forceinline__ float weight_of(const LayerMatrices &m, int e, int k, int n) {
    if (m.kind == LAYER_F32) {
        const float *mat = (const float *)m.data + e * m.stride;
        return m.trans ? mat[n * m.ld + k] : mat[k * m.ld + n];
    }
    if (m.kind == LAYER_F8) {
        const unsigned char *w = (const unsigned char *)m.data + e * m.f8.bytes;
        const unsigned code = w[(k / kF8Block * m.f8.rows + n) * kF8Block +
                                f8_place(k % kF8Block / 16, n) + k % 16];
        return __builtin_amdgcn_cvt_f32_fp8(code, 0) *
               ((const float *)(w + m.f8.planes))[k / kF8Block * m.f8.cols + n / kF8Block];
    }
    const W4Layout &l = m.w4;
    const unsigned char *rec = (const unsigned char *)m.data + e * l.expert_bytes +
                               n / kW4Cols * l.strip_bytes + (int64_t)(k / kW4Block) * l.record;
    const int col = n % kW4Cols, kk = k % kW4Block;
    const unsigned word =
        *(const unsigned *)(rec + 16 * (16 * w4_part(kk % 32) + col) + 4 * (kk / 32));
    const int part = col * l.parts + kk / (kW4Block / l.parts);
    const int z = l.zeros ? rec[kW4Codes + l.parts * kW4Cols * l.scale_size + part] : 8;
    return (float)((int)(word >> w4_shift(w4_index(kk % 32)) & 15) - z) *
           w4_scale(rec + kW4Codes + part * l.scale_size, l.scale_type);
}

// A work-item for each element of h, or of y.
__global__ __launch_bounds__(256) void layer_up_short_kernel(LayerProblem p, Hidden o) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t q = blockIdx.y; q < (int64_t)p.tokens * p.top; q += gridDim.y) {
        const int64_t t = q / p.top;
        const int e = p.ids[t * p.ldids + q % p.top];
        if (n >= p.hidden || e < 0 || e >= p.experts) continue;
        float z = 0.0f, u = 0.0f;
        for (int k = 0; k < p.width; ++k) {
            const float x = p.x[t * p.ldx + k];
            u = fmaf(x, weight_of(p.up, e, k, (int)n), u);
            if (p.gated) z = fmaf(x, weight_of(p.gate, e, k, (int)n), z);
        }
        o.h[q * o.ld + n] = p.gated ? activate(z, p.act) * u : activate(u, p.act);
    }
}
__global__ __launch_bounds__(256) void layer_down_short_kernel(LayerProblem p, Hidden o) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t t = blockIdx.y; t < p.tokens; t += gridDim.y) {
        if (n >= p.width) continue;
        float sum = 0.0f;
        for (int j = 0; j < p.top; ++j) {
            const int e = p.ids[t * p.ldids + j];
            if (e < 0 || e >= p.experts) continue;
            float back = 0.0f;
            for (int k = 0; k < p.hidden; ++k)
                back = fmaf(o.h[(t * p.top + j) * o.ld + k], weight_of(p.down, e, k, (int)n), back);
            sum = fmaf(p.weights[t * p.ldw + j], back, sum);
        }
        p.y[t * p.ldy + n] = sum;
    }
}

// ---------------------------------------------------------------------------------------------------

hipError_t launch_short(void (*kernel)(LayerProblem, Hidden), const LayerProblem &p, const Hidden &o,
                        int64_t rows, int64_t cols, hipStream_t s) {
    const int64_t x = (cols + 255) / 256, most = most_groups(256) / x;
    const int64_t y = rows < 65535 ? rows : 65535;
    if (most < 1) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    return launch(kernel, dim3((unsigned)x, (unsigned)(y < most ? y : most)), dim3(256), 0, s, p, o);
}

// Items that there can be.
int64_t most_items(const LayerProblem &p, int mr) {
    return most_blocks(p.tokens * p.top, p.experts, mr);
}

template <class E, bool GATED, int W, int D>
hipError_t launch_up_with(const LayerProblem &p, const Hidden &o, hipStream_t s) {
    const int64_t strips = ((int64_t)p.hidden + E::COLS - 1) / E::COLS, items = most_items(p, E::MR);
    if (strips > most_groups(64 * W) / items) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    return launch(layer_up_kernel<E, GATED, W, D>, dim3((unsigned)(strips * items)), dim3(64 * W), 0, s,
                  p, o, (int)items);
}

template <class E, int W>
DownLds<E, W> down_lds_of(const LayerProblem &p, const Hidden &o) {
    const int items = (int)most_items(p, E::MR);
    return {p.tokens, items, o.offsets != nullptr ? p.tokens * p.top : items * E::MR};
}

constexpr int kLds = 160 * 1024;

template <class E, int W, int D>
hipError_t launch_down_with(const LayerProblem &p, const Hidden &o, hipStream_t s, int split = 1) {
    const int64_t strips = ((int64_t)p.width + E::COLS - 1) / E::COLS;
    const DownLds<E, W> lds = down_lds_of<E, W>(p, o);
    if (strips > most_groups(64 * W) / split || lds.bytes() > kLds) return hipErrorInvalidValue;
    if (p.check) return hipSuccess;
    const hipError_t st = launch(layer_down_kernel<E, W, D>, dim3((unsigned)(strips * split)),
                                 dim3(64 * W), (size_t)lds.bytes(), s, p, o, lds.items, lds.list, split);
    if (st != hipSuccess || split == 1) return st;
    const int64_t groups = ((int64_t)p.tokens * p.width + 255) / 256;
    return launch(layer_join_kernel, dim3((unsigned)(groups < 65536 ? groups : 65536)), dim3(256), 0, s,
                  p, o, split);
}

// STRIPS of G and as many of U, or twice as many of U alone, on four waves.
template <class R, class F, int STRIPS, int D>
hipError_t launch_up_as(const LayerProblem &p, const Hidden &o, hipStream_t s) {
    return p.gated ? launch_up_with<CodesEngine<R, F, 2, STRIPS>, true, 4, D>(p, o, s)
                   : launch_up_with<CodesEngine<R, F, 1, 2 * STRIPS>, false, 4, D>(p, o, s);
}

// The rows that an expert has on average.
int64_t rows_each(const LayerProblem &p) {
    return ((int64_t)p.tokens * p.top + p.experts - 1) / p.experts;
}

// The form by the rows that an expert has on average.  More strips cut a row's values once for
// more columns, fewer leave more registers for loads in flight.  Times in us, back to back,
// two sets of weights in turn, gated, MR rows by STRIPS strips of each matrix, on four (eight)
// waves:
//   tokens top of experts, width, hidden       2 x 1        5 x 2      10 x 2      16 x 1     16 x 2
//    1, 8 of 64, 2048, 1408, 8 bits          10.5 (12.1)  11.5        14.1 (17.0)  15.0       14.2
//    1, 2 of  8, 4096, 4096, 4 bits          10.6 (10.6)  13.9        17.6 (14.5)  16.8       15.1
//    4, 8 of 64, 2048, 1408, 8 bits          30.9 (39)    36.0             (46)    45         37
//   16, 2 of  8, 4096, 4096, 4 bits            64 (85)      45 (60)     72 (58)    62 (80)    46 (55)
//   16, 2 of  8, 4096, 4096, 8 bits            74 (94)      64 (73)     58 (65)    70 (84)    53 (66)
//   32, 4 of 16, 4096, 1408, 8 bits            82           56 (64)     48 (55)    55 (72)    47 (59)
//   64, 4 of 16, 4096, 1408, 8 bits           140           88 (101)    66 (79)    79 (94)    62 (73)
//   64, 4 of 16, 2048, 1408, 4 bits            79           38 (56)     54 (45)    38 (50)    30 (38)
// (16 x 4 on four waves: 48, 54, 46, 64 and 39 in the last five lines; on two waves nothing gains.)
template <class F>
hipError_t launch_up(const LayerProblem &p, const Hidden &o, hipStream_t s) {
    if (rows_each(p) <= 2) return launch_up_as<Rows<1>, F, 1, 2>(p, o, s);
    return launch_up_as<Rows<8>, F, 2, 1>(p, o, s);
}

// The CUs that shares of y are to fill: a number, since the size of the workspace goes by it.
constexpr int kCus = 256, kSplit = 16;

// Work-groups that share a strip of y: as many as bring their number to `groups`, each with a
// block of k for each of its waves at least.
int shares(const LayerProblem &p, int cols, int mr, int block, int waves, int64_t groups) {
    const int64_t strips = ((int64_t)p.width + cols - 1) / cols;
    const int64_t units = most_items(p, mr) * (((int64_t)p.hidden + block - 1) / block);
    int64_t n = groups / strips;
    if (n > units / waves) n = units / waves;
    return (int)(n < 1 ? 1 : n < kSplit ? n : kSplit);
}

// STRIPS strips of y for each work-group, or two where the LDS does not hold the sums of more (it
// holds those of two with the tables of any choices).
template <class R, class F, int STRIPS>
hipError_t launch_down_as(const LayerProblem &p, const Hidden &o, int64_t groups, hipStream_t s) {
    using E = CodesEngine<R, F, 1, STRIPS>;
    if constexpr (STRIPS > 2) {
        if (down_lds_of<E, 8>(p, o).bytes() > kLds)
            return launch_down_as<R, F, 2>(p, o, groups, s);
    } else {
        constexpr int pairs = kLayerTokens * kLayerTop;
        static_assert(DownLds<E, 8>{kLayerTokens, pairs, pairs}.bytes() <= kLds, "any choices");
    }
    return launch_down_with<E, 8, 1>(p, o, s, shares(p, E::COLS, E::MR, E::BLOCK, 8, groups));
}

// Likewise; where few pairs or columns leave few work-groups, several share a strip's items and a
// third kernel adds what they have (about 3 us).  One token's choices go without, on
// sixteen waves each.  Times in us, MR rows by STRIPS strips, by the work-groups for each CU:
//   tokens top of experts, hidden, width          1/4    1/2     1      2      4
//    1, 8 of 64, 1408, 2048, 8 bits,  2 x 2             16.9   12.8   11.4          (sixteen waves, 2 x 1: 12.2)
//    1, 2 of  8, 4096, 4096, 4 bits,  2 x 2             12.7   11.2   11.3          (sixteen waves, 2 x 1:  9.8)
//    4, 8 of 64, 1408, 2048, 8 bits,  2 x 2     45     31     23     25     33
//   16, 2 of  8, 4096, 4096, 4 bits,  2 x 2            82     51     41     48
//   16, 2 of  8, 4096, 4096, 4 bits,  5 x 2            55     37     32     40
//   16, 2 of  8, 4096, 4096, 4 bits, 16 x 4     80     49     34     43
//   16, 2 of  8, 4096, 4096, 8 bits, 16 x 4     71     46     36     47
//   32, 4 of 16, 1408, 4096, 8 bits, 16 x 4     64     44     34     49
//   64, 4 of 16, 1408, 4096, 8 bits, 16 x 4     94     60     43     60     91
//   64, 4 of 16, 1408, 4096, 8 bits, 16 x 2            74     50     51     63
//   64, 4 of 16, 1408, 2048, 4 bits, 16 x 4     60     41     33     48
// (The last four lines with items found one by one; as they are found now about 7 less each.
// A second block in flight, for 217 registers: 46 instead of 42 in the 8-bit line before them.)
template <class F>
hipError_t launch_down(const LayerProblem &p, const Hidden &o, hipStream_t s) {
    if (rows_each(p) > 2) return launch_down_as<Rows<8>, F, 4>(p, o, kCus, s);
    if (p.tokens > 1) return launch_down_as<Rows<1>, F, 2>(p, o, kCus, s);
    return launch_down_with<CodesEngine<Rows<1>, F, 1, 1>, 16, 2>(p, o, s);
}

// h, after it the arrays of the sort and the shares of y, in bytes.
struct Workspace {
    int64_t ld;
    __int128 h, offsets, pairs, sort, parts;
    __int128 before_parts() const { return h + offsets + 2 * pairs + sort; }
    __int128 bytes() const { return before_parts() + parts; }
};

Workspace workspace_of(int tokens, int top, int experts, int width, int hidden) {
    auto whole = [](__int128 b) { return (b + 15) / 16 * 16; };
    Workspace w{};
    const int64_t n = (int64_t)tokens * top;
    w.ld = ((int64_t)hidden + 3) / 4 * 4;
    w.h = (__int128)n * w.ld * 4;
    if (n > 64) {
        w.offsets = whole(((__int128)experts + 1) * 4);
        w.pairs = whole((__int128)n * 4);
        w.sort = whole(route_workspace({tokens, top}, experts));
    }
    // at most so many shares of y (shares(); a work-group has 16 columns at least)
    const int64_t strips = ((int64_t)width + 15) / 16, most = 4 * kCus / strips;
    const int64_t split = most < kSplit ? most : kSplit;
    if (split > 1) w.parts = (__int128)split * tokens * width * 4;
    return w;
}

// Shares as above (5 tokens, 3 of 7 experts of 1531 x 1021: 98 us by one work-group a strip, 33 by
// four, 21 by sixteen).  Eight waves' sums of 64 columns for more tokens would leave the LDS
// too little.
template <bool TB>
hipError_t launch_down_plain(const LayerProblem &p, const Hidden &o, hipStream_t s) {
    using E = PlainEngine<TB, 1>;
    const int waves = p.tokens <= 16 ? 8 : 4;
    const int n = shares(p, E::COLS, E::MR, E::BLOCK, waves, kCus);
    return waves == 8 ? launch_down_with<E, 8, 1>(p, o, s, n) : launch_down_with<E, 4, 1>(p, o, s, n);
}

// One round: all tokens of p.
hipError_t launch_round(const LayerProblem &p, hipStream_t s) {
    const Workspace w = workspace_of(p.tokens, p.top, p.experts, p.width, p.hidden);
    Hidden o{(float *)p.workspace, w.ld, nullptr, nullptr,
             (float *)(p.workspace + (int64_t)w.before_parts())};
    hipError_t st = hipSuccess;
    const bool short_up = p.width < 4 || (p.up.kind == LAYER_F32 && p.hidden < 4);
    const bool short_down = p.hidden < 4 || (p.down.kind == LAYER_F32 && p.width < 4);
    if (p.tokens * p.top > 64 && !(short_up && short_down)) {
        int *offsets = (int *)(p.workspace + (int64_t)w.h);
        int *order = (int *)((unsigned char *)offsets + (int64_t)w.offsets);
        int *position = (int *)((unsigned char *)order + (int64_t)w.pairs);
        if (!p.check)
            st = launch_route_sort({p.tokens, p.top}, p.experts, p.ids, p.ldids, offsets, order,
                                   position, (unsigned char *)position + (int64_t)w.pairs, s);
        if (st != hipSuccess) return st;
        o.offsets = offsets;
        o.order = order;
    }
    if (short_up)
        st = launch_short(layer_up_short_kernel, p, o, (int64_t)p.tokens * p.top, p.hidden, s);
    else if (p.up.kind == LAYER_F32 && p.up.trans)
        st = p.gated ? launch_up_with<PlainEngine<true, 2>, true, 8, 1>(p, o, s)
                     : launch_up_with<PlainEngine<true, 1>, false, 8, 1>(p, o, s);
    else if (p.up.kind == LAYER_F32)
        st = p.gated ? launch_up_with<PlainEngine<false, 2>, true, 8, 1>(p, o, s)
                     : launch_up_with<PlainEngine<false, 1>, false, 8, 1>(p, o, s);
    else if (p.up.kind == LAYER_F8)
        st = launch_up<EightBits>(p, o, s);
    else
        st = p.up.w4.parts == 4   ? launch_up<FourBits<4>>(p, o, s)
             : p.up.w4.parts == 2 ? launch_up<FourBits<2>>(p, o, s)
                                  : launch_up<FourBits<1>>(p, o, s);
    if (st != hipSuccess) return st;
    if (short_down) return launch_short(layer_down_short_kernel, p, o, p.tokens, p.width, s);
    if (p.down.kind == LAYER_F32)
        return p.down.trans ? launch_down_plain<true>(p, o, s) : launch_down_plain<false>(p, o, s);
    if (p.down.kind == LAYER_F8) return launch_down<EightBits>(p, o, s);
    return p.down.w4.parts == 4   ? launch_down<FourBits<4>>(p, o, s)
           : p.down.w4.parts == 2 ? launch_down<FourBits<2>>(p, o, s)
                                  : launch_down<FourBits<1>>(p, o, s);
}

}  // namespace

__int128 layer_workspace(int tokens, int top, int experts, int width, int hidden) {
    if (tokens == 0 || top == 0 || experts == 0 || width == 0 || hidden == 0) return 0;
    return workspace_of(tokens < kLayerTokens ? tokens : kLayerTokens, top, experts, width, hidden)
        .bytes();
}

hipError_t launch_layer(const LayerProblem &given, hipStream_t s) {
    LayerProblem p = given;
    if (p.top == 0 || p.experts == 0 || p.hidden == 0) {
        p.top = 0;  // nothing is added
        return launch_short(layer_down_short_kernel, p, Hidden{}, p.tokens, p.width, s);
    }
    // A call that one of its launches refuses enqueues nothing: full rounds and the last one are
    // looked at first.
    p.check = true;
    for (const int n : {kLayerTokens, given.tokens % kLayerTokens}) {
        p.tokens = n;
        const hipError_t st = n == 0 || n > given.tokens ? hipSuccess : launch_round(p, s);
        if (st != hipSuccess) return st;
    }
    p.check = false;
    // rounds on one stream follow each other and can share the workspace
    for (int t = 0; t < given.tokens; t += kLayerTokens) {
        p.tokens = given.tokens - t < kLayerTokens ? given.tokens - t : kLayerTokens;
        p.ids = given.ids + t * given.ldids;
        p.weights = given.weights + t * given.ldw;
        p.x = given.x + t * given.ldx;
        p.y = given.y + t * given.ldy;
        const hipError_t st = launch_round(p, s);
        if (st != hipSuccess) return st;
    }
    return hipSuccess;
}

}  // namespace sgemm
