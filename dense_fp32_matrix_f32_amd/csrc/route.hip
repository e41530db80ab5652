// route.hip -- the order of rows by expert, and rows moved along it.
//
// All of it is bound by memory traffic (or, for a few tokens, by the launch).  The
// pairs (token, choice) are numbered f = token * top + choice.
#include <type_traits>

#include "experts.h"
#include "groups.h"

namespace sgemm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// ---------------------------------------------------------------------------
// The order: a counting sort by expert, stable in f.  Dropped pairs count as one
// more expert after the others, whose places are written as -1.
//
// The pairs are cut into chunks, one for each work-group, and a chunk into equal
// runs, one for each wave.  A work-group counts its chunk's pairs by expert and
// wave in LDS; adding the counts of the chunks before it and of all smaller experts
// gives the place of each wave's first pair of each expert, and a wave then walks
// its run 64 pairs at a time, a pair's rank among equal ones found by comparing
// the bits of its expert with ballots.  With more than one chunk a first kernel
// leaves every chunk's counts in the workspace.  No place depends on which
// work-group or wave runs first.  262144 pairs for 256 experts: 3.3 + 11.2 us (one
// work-group for each expert, walking all pairs: 344 us); eight pairs: 2.6 us, the time of
// a launch.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortChunks = 128;         // at most
constexpr int kSortBuckets = 896;        // at most (63 KB of LDS)

// Work-items that add up the counts of one bucket.
__host__ __device__ constexpr int sort_slices(int buckets) { return kSortThreads / buckets; }

struct SortArgs {
    Pairs p;
    int experts;
    const int *ids;
    int64_t ldids;
    int run;     // pairs of a wave (a multiple of 64)
    int chunks;
    int *counts;  // chunks x buckets, or NULL with one chunk
    int buckets;  // experts + 1, or of a digit
    // sorting by digits only:
    const int *from;  // the pairs in the order of the digits below, or NULL: by number
    int below;        // what the digits below count to
};

__device__ __forceinline__ int expert_of(const SortArgs &a, int f) {
    const int e = a.ids[(int64_t)(f / a.p.top) * a.ldids + f % a.p.top];
    return e < 0 || e >= a.experts ? a.experts : e;
}

// The pair that is the i-th to be sorted, and a pair's bucket.
template <bool DIGITS>
__device__ __forceinline__ int pair_at(const SortArgs &a, int i) {
    return DIGITS && a.from != nullptr ? a.from[i] : i;
}
template <bool DIGITS>
__device__ __forceinline__ int bucket_of(const SortArgs &a, int f) {
    const int e = expert_of(a, f);
    return DIGITS ? e / a.below % a.buckets : e;
}

// The pairs of this wave (none, where its run starts past the last pair).
struct Run {
    int64_t begin, end;

    __device__ __forceinline__ explicit Run(const SortArgs &a) {
        const int64_t n = a.p.count();
        begin = min(((int64_t)blockIdx.x * kSortWaves + (threadIdx.x >> 6)) * a.run, n);
        end = min(begin + a.run, n);
    }
};

// The run's pairs by bucket, added to `mine`.
template <bool DIGITS>
__device__ __forceinline__ void count_run(const SortArgs &a, const Run &run, int *mine) {
    for (int64_t f = run.begin + (threadIdx.x & 63); f < run.end; f += 64)
        // sums of ones: any order gives the same
        atomicAdd(&mine[bucket_of<DIGITS>(a, pair_at<DIGITS>(a, (int)f))], 1);
}

template <bool DIGITS>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
    __shared__ int hist[kSortBuckets];
    const int buckets = a.buckets;
    for (int e = threadIdx.x; e < buckets; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    count_run<DIGITS>(a, Run(a), hist);
    __syncthreads();
    for (int e = threadIdx.x; e < buckets; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * buckets + e] = hist[e];
}

// By digits, offsets are not written, and without position (all digits but the last) order
// gets the dropped pairs too.
template <bool DIGITS>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a, int *offsets,
                                                                  int *order, int *position) {
    extern __shared__ int next[];  // [wave][bucket]: the place of the next pair
    __shared__ int sums[kSortWaves];
    const int buckets = a.buckets;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // the chunks' counts of a bucket, before this chunk and all, added by `slices`
    // work-items, each over every slices-th chunk
    int *parts = next + kSortWaves * buckets;  // [slice][bucket] of each
    const int slices = sort_slices(buckets);
    if (a.counts != nullptr && tid < slices * buckets) {
        const int slice = tid / buckets, *c = a.counts + tid % buckets;
        int before = 0, all = 0;
        for (int b0 = slice; b0 < a.chunks; b0 += 16 * slices) {
            int v[16];  // loads without a branch, so that all are in flight
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] = c[(int64_t)min(b0 + u * slices, a.chunks - 1) * buckets];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int b = b0 + u * slices;
                if (b < (int)blockIdx.x) before += v[u];
                if (b < a.chunks) all += v[u];
            }
        }
        parts[tid] = before;
        parts[slices * buckets + tid] = all;
    }
    for (int i = tid; i < buckets * kSortWaves; i += kSortThreads) next[i] = 0;
    __syncthreads();
    const Run run(a);
    int *mine = next + wave * buckets;
    count_run<DIGITS>(a, run, mine);
    __syncthreads();

    // one work-item for each bucket (kSortBuckets <= kSortThreads)
    int before = 0, all = 0;
    if (tid < buckets) {
        if (a.counts != nullptr) {
            for (int i = 0; i < slices; ++i) {
                before += parts[i * buckets + tid];
                all += parts[(slices + i) * buckets + tid];
            }
        } else {
            for (int w = 0; w < kSortWaves; ++w) all += next[w * buckets + tid];
        }
    }
    int upto = wave_scan(all);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += sums[w];
    if (tid < buckets) {
        const int first = upto - all;
        if (!DIGITS && blockIdx.x == 0) offsets[tid] = first;
        int at = first + before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = next[w * buckets + tid];
            next[w * buckets + tid] = at;
            at += c;
        }
    }
    __syncthreads();

    for (int64_t base = run.begin; base < run.end; base += 64) {
        const bool have = base + lane < run.end;
        const int f = have ? pair_at<DIGITS>(a, (int)(base + lane)) : 0;
        const int e = have ? bucket_of<DIGITS>(a, f) : buckets;
        // the lanes with the same bucket
        unsigned long long same = __ballot(have);
        for (int bit = 1; bit < buckets; bit *= 2) {
            const unsigned long long set = __ballot(e & bit);
            same &= e & bit ? set : ~set;
        }
        if (have) {
            const unsigned long long below = same & ((1ull << lane) - 1);
            const int at = mine[e] + __popcll(below);
            if (DIGITS && position == nullptr) {
                order[at] = f;
            } else {
                const bool kept = (DIGITS ? expert_of(a, f) : e) < a.experts;
                position[f] = kept ? at : -1;
                order[at] = kept ? f : -1;
            }
        }
        // the last lane of each bucket moves its place on, after all have read it
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have && (same >> lane) == 1) mine[e] += __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// More experts than fit LDS: the same stable sort by one digit of the expert's number
// after the other, the lowest first.  The digits have the smallest base that makes do
// with as few of them as possible.  What remains is where each expert's pairs begin,
// which a search of the order for its number gives.
struct Digits {
    int count, base;

    explicit Digits(int experts) : count(1), base(kSortBuckets) {
        const int64_t numbers = (int64_t)experts + 1;  // dropped pairs have the last
        while (power(base) < numbers) ++count;
        while (power(base - 1) >= numbers) --base;
    }
    int64_t power(int x) const {
        int64_t r = 1;
        for (int i = 0; i < count; ++i) r *= x;
        return r;
    }
};

__global__ __launch_bounds__(256) void sort_offsets_kernel(SortArgs a, const int *order,
                                                           int *offsets) {
    const int n = a.p.count();
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e <= a.experts;
         e += (int64_t)gridDim.x * 256) {
        int lo = 0, hi = n;  // the first place of an expert not below e
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2, f = order[mid];
            if ((f < 0 ? a.experts : expert_of(a, f)) < e)
                lo = mid + 1;
            else
                hi = mid;
        }
        offsets[e] = lo;
    }
}

// Few pairs for not many more experts than fit LDS, in one launch: one work-group for a
// bucket.  It counts the pairs of the buckets below its own, then walks all pairs in
// order and gives its own the places from there on, ranked by a ballot in a wave and a
// running sum over waves.
__global__ __launch_bounds__(kSortThreads) void sort_each_kernel(SortArgs a, int *offsets,
                                                                 int *order, int *position) {
    __shared__ int sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = a.p.count(), me = blockIdx.x;
    int below = 0;
    for (int f = tid; f < n; f += kSortThreads) below += expert_of(a, f) < me;
    for (int d = 32; d; d /= 2) below += __shfl_xor(below, d);
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    int place = 0;
    for (int w = 0; w < kSortWaves; ++w) place += sums[w];
    if (tid == 0) offsets[me] = place;
    __syncthreads();
    for (int base = 0; base < n; base += kSortThreads) {
        const int f = base + tid;
        const bool mine = f < n && expert_of(a, f) == me;
        const unsigned long long who = __ballot(mine);
        if (lane == 0) sums[wave] = __popcll(who);
        __syncthreads();
        int at = place;
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) at += sums[w];
            place += sums[w];
        }
        if (mine) {
            at += __popcll(who & ((1ull << lane) - 1));
            position[f] = me < a.experts ? at : -1;
            order[at] = me < a.experts ? f : -1;
        }
        __syncthreads();
    }
}

// Pairs of a wave and chunks.  Up to 6144 pairs are one chunk: a call with them takes 9.6
// us for 4 experts and 11.3 for 256, with two launches 13.3 and 13.5 (8192 pairs: 10.4 and
// 13.8 against 13.5).
void sort_cut(int64_t n, int *run, int *chunks) {
    const int64_t least = 384ll * kSortWaves;
    const int64_t even = (n + kSortChunks - 1) / kSortChunks;
    const int64_t chunk = n <= least ? n : even < 1024 ? 1024 : even;
    *run = (int)((chunk + kSortThreads - 1) / kSortThreads * 64);
    const int64_t per = (int64_t)*run * kSortWaves;
    *chunks = n > 0 ? (int)((n + per - 1) / per) : 1;
}

// Whether a work-group for each bucket takes the call instead of the digits.  Times of a
// call / of its kernels in us:
//   pairs, experts       each bucket     digits
//      8,    896          10 /   6      17 /   9
//   6144,    896          21 /  21      36 /  36
//   6144,   1536          32 /  32      37 /  37
//   4096,   2048          29 /  29      29 /  28
//   1024,   3000          17 /  17      18 /  15
//   2048,   3000          24 /  24      20 /  20
//      8,   4096          17 /  17      17 /  10
//   1024,   4096          23 /  22      17 /  15
//   8192,   1024          30 /  30      27 /  25
// and 262144 pairs for 1024 experts 830 against 38 (22 for 895 experts in one pass),
// 2^20 pairs for 2^20 experts 178 in three digits.
bool sort_each(int64_t n, int chunks, int experts) {
    return chunks == 1 && experts * (n + 4096) <= 1 << 24;
}

// ---------------------------------------------------------------------------
// Rows there and back.  The lanes of a row take four columns each (16-byte accesses,
// which gfx950 takes at any multiple of four bytes).  8192 tokens of 2048 columns with
// four choices each: gather 56 us (335 MB, 6.0 TB/s, mostly written), combine 58 us (335
// MB, 5.8 TB/s, mostly read), the gradients 128 us (603 MB, 4.7 TB/s; a copy of 2 GiB
// reaches 5.0); what one kernel leaves in the last cache to be written back is part of
// the next one's time, so the four calls of a step together count: 301 us.  Two column
// vectors of a lane in flight instead of one changed nothing.

// Work-items for a row: enough for its vectors, a power of two from 16 to `most`.
int lanes_for(int width, int most) {
    int lanes = 16;
    while (lanes < most && lanes * 4 < width) lanes *= 2;
    return lanes;
}

// Calls body(c, vector) for this lane's columns of [begin, end): with 16-byte vectors
// at c, then for the last end % 4 columns one by one on the first lanes.
template <class Body>
__device__ __forceinline__ void for_columns(int64_t begin, int64_t end, int lane, int lanes,
                                            const Body &body) {
    const int64_t whole = begin + (end - begin) / 4 * 4;
    for (int64_t c = begin + 4 * lane; c < whole; c += 4 * lanes) body(c, std::true_type{});
    if (lane < end - whole) body(whole + lane, std::false_type{});
}

template <bool VECTOR>
using Cols = typename std::conditional<VECTOR, f32x4, float>::type;

__device__ __forceinline__ f32x4 load(const float *p, std::true_type) {
    return *(const f32x4_any *)p;
}
__device__ __forceinline__ float load(const float *p, std::false_type) { return *p; }
template <bool PAST = false>
__device__ __forceinline__ void store(float *p, f32x4 v) {
    if constexpr (PAST)
        __builtin_nontemporal_store((f32x4_any)v, (f32x4_any *)p);
    else
        *(f32x4_any *)p = v;
}
template <bool PAST = false>
__device__ __forceinline__ void store(float *p, float v) {
    if constexpr (PAST)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
__device__ __forceinline__ f32x4 mul_add(float w, f32x4 v, f32x4 sum) {
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(w, v[e], sum[e]);
    return sum;
}
__device__ __forceinline__ float mul_add(float w, float v, float sum) { return fmaf(w, v, sum); }
__device__ __forceinline__ float dot_add(f32x4 a, f32x4 b, float sum) {
    for (int e = 0; e < 4; ++e) sum = fmaf(a[e], b[e], sum);
    return sum;
}
__device__ __forceinline__ float dot_add(float a, float b, float sum) { return fmaf(a, b, sum); }

// Loads of what is read once, past the caches: gather, combine, gradients and combine
// of 4096 tokens of 2048 columns with four choices 155 -> 146 us, of 8192 tokens 339 ->
// 268 with buffers allocated once and 339 -> 326 with new ones.
__device__ __forceinline__ f32x4 load_once(const float *p, std::true_type) {
    return __builtin_nontemporal_load((const f32x4_any *)p);
}
__device__ __forceinline__ float load_once(const float *p, std::false_type) {
    return __builtin_nontemporal_load(p);
}

constexpr int J = 4;  // choices whose loads are in flight together

// Places and weights of choices j0 .. j0+3 of a token; -1 past the last and where
// there is none.
struct Choices {
    int place[J];
    float w[J];

    __device__ __forceinline__ Choices(Pairs p, int64_t t, int j0, const int *position,
                                       const float *weights, int64_t ldw) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = j0 + j < p.top ? position[t * p.top + j0 + j] : -1;
            place[j] = at >= 0 && at < p.count() ? at : -1;
            w[j] = j0 + j < p.top && weights != nullptr ? weights[t * ldw + j0 + j] : 1.0f;
        }
    }
    // A row to load from without a branch: a choice without a place reads row 0, and
    // what it reads is not used.
    __device__ __forceinline__ int64_t row(int j) const { return place[j] >= 0 ? place[j] : 0; }
};

// rows[position[t, j]] = x[t]: a token's row is read once and written to its places.
// The grid's second axis cuts the columns into pieces of `span`.
__global__ __launch_bounds__(256) void gather_kernel(Pairs p, int width, int lanes, int span,
                                                     const int *__restrict__ position,
                                                     const float *__restrict__ x, int64_t ldx,
                                                     float *__restrict__ rows, int64_t ldrows) {
    const int per = 256 / lanes, lane = threadIdx.x % lanes;
    const int64_t begin = (int64_t)blockIdx.y * span, end = min((int64_t)width, begin + span);
    for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes; t < p.tokens;
         t += (int64_t)gridDim.x * per)
        for (int j0 = 0; j0 < p.top; j0 += J) {
            const Choices k(p, t, j0, position, nullptr, 0);
            for_columns(begin, end, lane, lanes, [&](int64_t c, auto vector) {
                const auto v = load(x + t * ldx + c, vector);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (k.place[j] >= 0) store(rows + k.place[j] * ldrows + c, v);
            });
        }
}

// Whether results are stored past the caches too: where the rows alone fill the last
// cache (256 MB), so that what is written takes the place of what is still to be read.
// The four calls above, in us:
//                                                        cached  past
//   8192 tokens of 2048, four choices (268 MB), new buffers  326   301
//   the same, buffers allocated once                         265   282
//   9000 tokens of 2048, four choices                        289   312
//   8192 tokens of 4096, two choices                         389   367
//   16384 tokens of 2048, four choices                       597   589
//   32768 tokens of 2048, eight choices                     2370  2251
//   4096 tokens of 2048, four choices (134 MB)               146   165
// (with new buffers the bound helps at 268 MB; buffers that stay, and sizes a little past
// it, lose 6 to 8%, larger ones and wider rows gain again)
bool store_past(Pairs p, int width) {
    return (int64_t)p.count() * width * 4 >= (int64_t)256 << 20;
}

// out[t] = sum of weights[t, j] * rows[position[t, j]] in the order of j.
template <bool PAST>
__global__ __launch_bounds__(256) void combine_kernel(Pairs p, int width, int lanes, int span,
                                                      const int *__restrict__ position,
                                                      const float *__restrict__ weights,
                                                      int64_t ldw, const float *__restrict__ rows,
                                                      int64_t ldrows, float *__restrict__ out,
                                                      int64_t ldout) {
    const int per = 256 / lanes, lane = threadIdx.x % lanes;
    const int64_t begin = (int64_t)blockIdx.y * span, end = min((int64_t)width, begin + span);
    for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes; t < p.tokens;
         t += (int64_t)gridDim.x * per) {
        const Choices first(p, t, 0, position, weights, ldw);
        for_columns(begin, end, lane, lanes, [&](int64_t c, auto vector) {
            Cols<decltype(vector)::value> sum = {};
            auto add = [&](const Choices &k) {
                Cols<decltype(vector)::value> v[J];
#pragma unroll
                for (int j = 0; j < J; ++j) v[j] = load_once(rows + k.row(j) * ldrows + c, vector);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (k.place[j] >= 0) sum = mul_add(k.w[j], v[j], sum);
            };
            if (p.top > 0) add(first);
            for (int j0 = J; j0 < p.top; j0 += J) add(Choices(p, t, j0, position, weights, ldw));
            store<PAST>(out + t * ldout + c, sum);
        });
    }
}

// The gradients of a token, four choices at a time: its dout is read once for them;
// a choice's product with its row is added over the lanes in a fixed order (a
// butterfly in each wave, then the waves in turn).
template <bool PAST>
__global__ __launch_bounds__(1024) void combine_grad_kernel(
    Pairs p, int width, int lanes, const int *__restrict__ position,
    const float *__restrict__ weights, int64_t ldw, const float *__restrict__ rows, int64_t ldrows,
    const float *__restrict__ dout, int64_t lddout, float *__restrict__ drows, int64_t lddrows,
    float *__restrict__ dweights) {
    __shared__ float part[16][J];
    const int per = blockDim.x / lanes, lane = threadIdx.x % lanes;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < p.tokens; t0 += (int64_t)gridDim.x * per) {
        const int64_t token = t0 + threadIdx.x / lanes;
        const bool have = token < p.tokens;  // every work-item reaches the barriers
        const int64_t t = have ? token : 0;
        for (int j0 = 0; j0 < p.top; j0 += J) {
            const Choices k(p, t, j0, position, weights, ldw);
            float dot[J] = {};
            if (have) {
                for_columns(0, width, lane, lanes, [&](int64_t c, auto vector) {
                    typedef Cols<decltype(vector)::value> V;
                    const V g = load(dout + t * lddout + c, vector);
                    if (dweights != nullptr) {
                        V y[J];
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            y[j] = load_once(rows + k.row(j) * ldrows + c, vector);
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            if (k.place[j] >= 0) dot[j] = dot_add(g, y[j], dot[j]);
                    }
                    if (drows != nullptr) {
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            if (k.place[j] >= 0)
                                store<PAST>(drows + k.place[j] * lddrows + c, k.w[j] * g);
                    }
                });
            }
            if (dweights == nullptr) continue;
#pragma unroll
            for (int j = 0; j < J; ++j)
                for (int d = min(lanes, 64) / 2; d > 0; d /= 2) dot[j] += __shfl_xor(dot[j], d);
            if (lanes > 64) {
                const int wave = threadIdx.x >> 6;
                __syncthreads();  // the last four choices' sums have been read
                if ((threadIdx.x & 63) == 0) {
#pragma unroll
                    for (int j = 0; j < J; ++j) part[wave][j] = dot[j];
                }
                __syncthreads();
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        for (int i = 1; i < lanes / 64; ++i) dot[j] += part[wave + i][j];
                }
            }
            if (have && lane == 0) {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (j0 + j < p.top)
                        dweights[t * ldw + j0 + j] = k.place[j] >= 0 ? dot[j] : 0.0f;
            }
        }
    }
}

// Work-groups of a launch; further tokens and buckets are taken in turn (1024
// work-items each stay below 2^32).
unsigned route_groups(int64_t groups) {
    return (unsigned)(groups < (1 << 21) ? groups : 1 << 21);
}

// Columns of a work-group's piece: all of them, or with too few tokens to fill the
// chip pieces of one vector a lane.
int span_for(int64_t groups, int width, int lanes) {
    if (groups >= 1024) return width;
    // the grid's second axis ends at 65535
    const int64_t least = ((int64_t)width + 65534) / 65535, vector = 4ll * lanes;
    return (int)((least + vector - 1) / vector * vector);
}

}  // namespace

size_t route_workspace(Pairs p, int experts) {
    int run, chunks;
    sort_cut(p.count(), &run, &chunks);
    if (experts < kSortBuckets)
        return chunks > 1 ? sizeof(int) * chunks * (size_t)(experts + 1) : 0;
    if (sort_each(p.count(), chunks, experts)) return 0;
    // the counts, and the pairs between two digits
    const size_t counts = chunks > 1 ? (size_t)chunks * Digits(experts).base : 0;
    return sizeof(int) * (counts + (size_t)p.count());
}

namespace {

// One pass of the sort.
template <bool DIGITS>
hipError_t launch_sort_pass(SortArgs a, int *offsets, int *order, int *position, hipStream_t s) {
    size_t lds = sizeof(int) * kSortWaves * (size_t)a.buckets;
    if (a.chunks == 1) {
        a.counts = nullptr;
    } else {
        lds += 2 * sizeof(int) * sort_slices(a.buckets) * (size_t)a.buckets;
        const hipError_t e = launch(sort_count_kernel<DIGITS>, dim3((unsigned)a.chunks),
                                    dim3(kSortThreads), 0, s, a);
        if (e != hipSuccess) return e;
    }
    return launch(sort_place_kernel<DIGITS>, dim3((unsigned)a.chunks), dim3(kSortThreads), lds, s,
                  a, offsets, order, position);
}

}  // namespace

hipError_t launch_route_sort(Pairs p, int experts, const int *ids, int64_t ldids, int *offsets,
                             int *order, int *position, void *workspace, hipStream_t s) {
    SortArgs a{p, experts, ids, ldids, 0, 0, (int *)workspace, experts + 1, nullptr, 1};
    sort_cut(p.count(), &a.run, &a.chunks);
    if (experts < kSortBuckets) return launch_sort_pass<false>(a, offsets, order, position, s);
    if (sort_each(p.count(), a.chunks, experts))
        return launch(sort_each_kernel, dim3((unsigned)experts + 1), dim3(kSortThreads), 0, s, a,
                      offsets, order, position);
    if (p.count() > 0) {
        const Digits digits(experts);
        a.buckets = digits.base;
        int *between = a.counts + (a.chunks > 1 ? (size_t)a.chunks * digits.base : 0);
        for (int left = digits.count - 1; left >= 0; --left) {
            // the last pass but one ends in `between`, the one before it in `order`
            int *to = left % 2 == 0 ? order : between;
            const hipError_t e = launch_sort_pass<true>(a, nullptr, to,
                                                        left == 0 ? position : nullptr, s);
            if (e != hipSuccess) return e;
            a.from = to;
            if (left > 0) a.below *= digits.base;
        }
    }
    const int64_t groups = ((int64_t)experts + 256) / 256;
    return launch(sort_offsets_kernel, dim3(route_groups(groups)), dim3(256), 0, s, a, order,
                  offsets);
}

hipError_t launch_route_gather(Pairs p, int width, const int *position, const float *x,
                               int64_t ldx, float *rows, int64_t ldrows, hipStream_t s) {
    const int lanes = lanes_for(width, 256);
    const int64_t groups = ((int64_t)p.tokens * lanes + 255) / 256;
    const int span = span_for(groups, width, lanes);
    const dim3 grid(route_groups(groups), (unsigned)(((int64_t)width + span - 1) / span));
    return launch(gather_kernel, grid, dim3(256), 0, s, p, width, lanes, span, position, x, ldx,
                  rows, ldrows);
}

hipError_t launch_route_combine(Pairs p, int width, const int *position, const float *weights,
                                int64_t ldw, const float *rows, int64_t ldrows, float *out,
                                int64_t ldout, hipStream_t s) {
    const int lanes = lanes_for(width, 256);
    const int64_t groups = ((int64_t)p.tokens * lanes + 255) / 256;
    const int span = span_for(groups, width, lanes);
    const dim3 grid(route_groups(groups), (unsigned)(((int64_t)width + span - 1) / span));
    return launch(store_past(p, width) ? combine_kernel<true> : combine_kernel<false>, grid,
                  dim3(256), 0, s, p, width, lanes, span, position, weights, ldw, rows, ldrows, out,
                  ldout);
}

hipError_t launch_route_combine_grad(Pairs p, int width, const int *position,
                                     const float *weights, int64_t ldw, const float *rows,
                                     int64_t ldrows, const float *dout, int64_t lddout,
                                     float *drows, int64_t lddrows, float *dweights,
                                     hipStream_t s) {
    // with few tokens a row gets up to 1024 work-items
    const int lanes = lanes_for(width, p.tokens < 512 ? 1024 : 256);
    const int threads = lanes > 256 ? lanes : 256;
    const int64_t groups = ((int64_t)p.tokens * lanes + threads - 1) / threads;
    return launch(store_past(p, width) ? combine_grad_kernel<true> : combine_grad_kernel<false>,
                  dim3(route_groups(groups)), dim3((unsigned)threads), 0, s, p, width, lanes,
                  position, weights, ldw, rows, ldrows, dout, lddout, drows, lddrows, dweights);
}

}  // namespace sgemm
