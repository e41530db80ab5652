// experts.h -- launchers behind include/sgemm_f32_experts.h (arguments already
// validated and non-empty).
#pragma once

#include "internal.h"

namespace sgemm {

struct Pairs {
    int tokens, top;
    __host__ __device__ int count() const { return tokens * top; }
};

size_t route_workspace(Pairs p, int experts);
hipError_t launch_route_sort(Pairs p, int experts, const int *ids, int64_t ldids, int *offsets,
                             int *order, int *position, void *workspace, hipStream_t s);
hipError_t launch_route_gather(Pairs p, int width, const int *position, const float *x,
                               int64_t ldx, float *rows, int64_t ldrows, hipStream_t s);
hipError_t launch_route_combine(Pairs p, int width, const int *position, const float *weights,
                                int64_t ldw, const float *rows, int64_t ldrows, float *out,
                                int64_t ldout, hipStream_t s);
hipError_t launch_route_combine_grad(Pairs p, int width, const int *position,
                                     const float *weights, int64_t ldw, const float *rows,
                                     int64_t ldrows, const float *dout, int64_t lddout,
                                     float *drows, int64_t lddrows, float *dweights,
                                     hipStream_t s);

// The products of groups.h's row ranges: C rows = alpha * A rows * op(B_e) + beta * C rows.
struct GroupedProblem {
    int rows, N, K, experts;
    const int *offsets;
    const float *A;
    int64_t lda;
    const float *B;
    int64_t ldb, strideb;
    float *C;
    int64_t ldc;
    bool tb;
    float alpha, beta;
};
hipError_t launch_grouped(const GroupedProblem &p, hipStream_t s);

// C_e (M x N) = alpha * A_e^T * D_e + beta * C_e over the rows of each expert.
struct GroupedTaProblem {
    int rows, M, N, experts;
    const int *offsets;
    const float *A;
    int64_t lda;
    const float *D;
    int64_t ldd;
    float *C;
    int64_t ldc, stridec;
    float alpha, beta;
};
hipError_t launch_grouped_ta(const GroupedTaProblem &p, hipStream_t s);

}  // namespace sgemm
