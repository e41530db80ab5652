// route.hip -- the order of rows by expert, and rows moved along it.
#include "experts.h"

namespace sgemm {

namespace {

constexpr int kSortThreads = 1024;

// One work-group for each expert: it counts the pairs of the experts below its
// own, then walks all pairs in order and gives its own the places from there on.
// A wave ranks its 64 pairs by a ballot, the work-group's waves by a running sum
// in LDS.  The group `experts` handles what is dropped, which has no places.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(Pairs p, int experts,
                                                            const int *__restrict__ ids,
                                                            int64_t ldids, int *offsets,
                                                            int *order, int *position) {
    constexpr int WAVES = kSortThreads / 64;
    __shared__ int sums[WAVES];
    const int me = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = p.count();
    auto id_of = [&](int f) {
        const int e = ids[(int64_t)(f / p.top) * ldids + f % p.top];
        return e < 0 || e >= experts ? experts : e;
    };
    int below = 0;
    for (int f = tid; f < n; f += kSortThreads) below += id_of(f) < me;
    for (int d = 32; d; d /= 2) below += __shfl_xor(below, d);
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    int next = 0;
    for (int w = 0; w < WAVES; ++w) next += sums[w];
    if (tid == 0) offsets[me] = next;
    __syncthreads();
    for (int base = 0; base < n; base += kSortThreads) {
        const int f = base + tid;
        const bool mine = f < n && id_of(f) == me;
        const unsigned long long who = __ballot(mine);
        if (lane == 0) sums[wave] = __popcll(who);
        __syncthreads();
        int at = next;
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) at += sums[w];
            next += sums[w];
        }
        if (mine) {
            at += __popcll(who & ((1ull << lane) - 1));
            position[f] = me < experts ? at : -1;
            order[at] = me < experts ? f : -1;
        }
        __syncthreads();
    }
}

// One work-group for each place (row) in turn.
__global__ __launch_bounds__(256) void gather_kernel(Pairs p, int width,
                                                     const int *__restrict__ order,
                                                     const float *__restrict__ x, int64_t ldx,
                                                     float *__restrict__ rows, int64_t ldrows) {
    const int n = p.count();
    for (int at = blockIdx.x; at < n; at += gridDim.x) {
        const int f = order[at];
        if (f < 0 || f >= n) continue;
        const float *from = x + (int64_t)(f / p.top) * ldx;
        float *to = rows + (int64_t)at * ldrows;
        for (int c = threadIdx.x; c < width; c += 256) to[c] = from[c];
    }
}

// One work-group for each token in turn.
__global__ __launch_bounds__(256) void combine_kernel(Pairs p, int width,
                                                      const int *__restrict__ position,
                                                      const float *__restrict__ weights,
                                                      int64_t ldw, const float *__restrict__ rows,
                                                      int64_t ldrows, float *__restrict__ out,
                                                      int64_t ldout) {
    const int n = p.count();
    for (int t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        for (int c = threadIdx.x; c < width; c += 256) {
            float sum = 0.0f;
            for (int j = 0; j < p.top; ++j) {
                const int at = position[(int64_t)t * p.top + j];
                if (at < 0 || at >= n) continue;
                const float w = weights ? weights[t * ldw + j] : 1.0f;
                sum = fmaf(w, rows[at * ldrows + c], sum);
            }
            out[t * ldout + c] = sum;
        }
    }
}

__global__ __launch_bounds__(256) void combine_grad_kernel(
    Pairs p, int width, const int *__restrict__ position, const float *__restrict__ weights,
    int64_t ldw, const float *__restrict__ rows, int64_t ldrows, const float *__restrict__ dout,
    int64_t lddout, float *__restrict__ drows, int64_t lddrows, float *__restrict__ dweights) {
    __shared__ float part[4];
    const int n = p.count();
    for (int f = blockIdx.x; f < n; f += gridDim.x) {
        const int t = f / p.top, j = f % p.top, at = position[f];
        const bool kept = at >= 0 && at < n;
        const float w = weights ? weights[t * ldw + j] : 1.0f;
        float dot = 0.0f;
        if (kept)
            for (int c = threadIdx.x; c < width; c += 256) {
                const float g = dout[t * lddout + c];
                if (drows) drows[at * lddrows + c] = w * g;
                if (dweights) dot = fmaf(g, rows[at * ldrows + c], dot);
            }
        for (int d = 32; d; d /= 2) dot += __shfl_xor(dot, d);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (dweights && threadIdx.x == 0)
            dweights[t * ldw + j] = ((part[0] + part[1]) + part[2]) + part[3];
        __syncthreads();
    }
}

unsigned grid_for(int64_t groups) { return (unsigned)(groups < 65536 ? groups : 65536); }

}  // namespace

size_t route_workspace(Pairs, int) { return 0; }

hipError_t launch_route_sort(Pairs p, int experts, const int *ids, int64_t ldids, int *offsets,
                             int *order, int *position, void *, hipStream_t s) {
    return launch(sort_kernel, dim3((unsigned)experts + 1), dim3(kSortThreads), 0, s, p, experts,
                  ids, ldids, offsets, order, position);
}

hipError_t launch_route_gather(Pairs p, int width, const int *order, const float *x, int64_t ldx,
                               float *rows, int64_t ldrows, hipStream_t s) {
    return launch(gather_kernel, dim3(grid_for(p.count())), dim3(256), 0, s, p, width, order, x,
                  ldx, rows, ldrows);
}

hipError_t launch_route_combine(Pairs p, int width, const int *position, const float *weights,
                                int64_t ldw, const float *rows, int64_t ldrows, float *out,
                                int64_t ldout, hipStream_t s) {
    return launch(combine_kernel, dim3(grid_for(p.tokens)), dim3(256), 0, s, p, width, position,
                  weights, ldw, rows, ldrows, out, ldout);
}

hipError_t launch_route_combine_grad(Pairs p, int width, const int *position,
                                     const float *weights, int64_t ldw, const float *rows,
                                     int64_t ldrows, const float *dout, int64_t lddout,
                                     float *drows, int64_t lddrows, float *dweights,
                                     hipStream_t s) {
    return launch(combine_grad_kernel, dim3(grid_for(p.count())), dim3(256), 0, s, p, width,
                  position, weights, ldw, rows, ldrows, dout, lddout, drows, lddrows, dweights);
}

}  // namespace sgemm
