// experts_api.hip -- the entry points of include/sgemm_f32_experts.h: argument
// validation on the host (before any HIP call) and launch on the caller's stream.
#include "sgemm_f32_experts.h"

#include <initializer_list>

#include "experts.h"
#include "extent.h"

using sgemm::Extent;
using sgemm::valid_size;

namespace {

int at_least_one(int x) { return x > 1 ? x : 1; }

// True if an array that is written meets another of the call.
bool any_overlap(std::initializer_list<Extent> written, std::initializer_list<Extent> read) {
    for (const Extent *w = written.begin(); w != written.end(); ++w) {
        for (const Extent &r : read)
            if (sgemm::overlaps(*w, r)) return true;
        for (const Extent *v = w + 1; v != written.end(); ++v)
            if (sgemm::overlaps(*w, *v)) return true;
    }
    return false;
}

Extent matrix(const void *p, int64_t rows, int64_t cols, int64_t ld) {
    return sgemm::extent(p, rows, cols, ld, 4);
}

Extent list(const void *p, int64_t n) { return sgemm::extent(p, 1, n, n, 4); }

constexpr Extent kNone{0, 0};  // meets nothing

bool valid_pairs(int tokens, int top) {
    return valid_size(tokens) && valid_size(top) && (int64_t)tokens * top <= sgemm::kMaxSize;
}

}  // namespace

extern "C" size_t sgemm_f32_route_workspace_size(int tokens, int top, int experts) {
    if (!valid_pairs(tokens, top) || !valid_size(experts)) return 0;
    return sgemm::route_workspace({tokens, top}, experts);
}

extern "C" hipError_t sgemm_f32_route_sort(int tokens, int top, int experts, const int *ids,
                                           int ldids, int *offsets, int *order, int *position,
                                           void *workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    if (!valid_pairs(tokens, top) || !valid_size(experts) || ldids < at_least_one(top) ||
        offsets == nullptr)
        return hipErrorInvalidValue;
    const int n = tokens * top;
    const Extent o = list(offsets, (int64_t)experts + 1);
    const size_t need = sgemm::route_workspace({tokens, top}, experts);
    if (n > 0) {
        if (ids == nullptr || order == nullptr || position == nullptr) return hipErrorInvalidValue;
        if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                         ((uintptr_t)workspace & 15) != 0))
            return hipErrorInvalidValue;
        const Extent ws = need > 0 ? sgemm::bytes_from(workspace, need) : kNone;
        if (any_overlap({o, list(order, n), list(position, n), ws},
                        {matrix(ids, tokens, top, ldids)}))
            return hipErrorInvalidValue;
    }
    return sgemm::launch_route_sort({tokens, top}, experts, ids, ldids, offsets, order, position,
                                    workspace, stream);
}

extern "C" hipError_t sgemm_f32_route_gather(int tokens, int top, int width, const int *position,
                                             const float *x, int ldx, float *rows, int ldrows,
                                             hipStream_t stream) {
    if (!valid_pairs(tokens, top) || !valid_size(width) || ldx < at_least_one(width) ||
        ldrows < at_least_one(width))
        return hipErrorInvalidValue;
    const int n = tokens * top;
    if (n == 0 || width == 0) return hipSuccess;
    if (position == nullptr || x == nullptr || rows == nullptr) return hipErrorInvalidValue;
    if (any_overlap({matrix(rows, n, width, ldrows)},
                    {list(position, n), matrix(x, tokens, width, ldx)}))
        return hipErrorInvalidValue;
    return sgemm::launch_route_gather({tokens, top}, width, position, x, ldx, rows, ldrows,
                                      stream);
}

extern "C" hipError_t sgemm_f32_route_combine(int tokens, int top, int width, const int *position,
                                              const float *weights, int ldw, const float *rows,
                                              int ldrows, float *out, int ldout,
                                              hipStream_t stream) {
    if (!valid_pairs(tokens, top) || !valid_size(width) || ldrows < at_least_one(width) ||
        ldout < at_least_one(width) || (weights != nullptr && ldw < at_least_one(top)))
        return hipErrorInvalidValue;
    const int n = tokens * top;
    if (tokens == 0 || width == 0) return hipSuccess;
    if (out == nullptr || (n > 0 && (position == nullptr || rows == nullptr)))
        return hipErrorInvalidValue;
    if (n > 0 &&
        any_overlap({matrix(out, tokens, width, ldout)},
                    {list(position, n), matrix(rows, n, width, ldrows),
                     weights != nullptr ? matrix(weights, tokens, top, ldw) : kNone}))
        return hipErrorInvalidValue;
    return sgemm::launch_route_combine({tokens, top}, width, position, weights, ldw, rows, ldrows,
                                       out, ldout, stream);
}

extern "C" hipError_t sgemm_f32_route_combine_grad(int tokens, int top, int width,
                                                   const int *position, const float *weights,
                                                   int ldw, const float *rows, int ldrows,
                                                   const float *dout, int lddout, float *drows,
                                                   int lddrows, float *dweights,
                                                   hipStream_t stream) {
    if (!valid_pairs(tokens, top) || !valid_size(width) || lddout < at_least_one(width) ||
        (dweights != nullptr && ldrows < at_least_one(width)) ||
        (drows != nullptr && lddrows < at_least_one(width)) ||
        ((weights != nullptr || dweights != nullptr) && ldw < at_least_one(top)))
        return hipErrorInvalidValue;
    const int n = tokens * top;
    if (n == 0 || (drows == nullptr && dweights == nullptr)) return hipSuccess;
    if (width == 0 && dweights == nullptr) return hipSuccess;
    if (position == nullptr ||
        (width > 0 && (dout == nullptr || (dweights != nullptr && rows == nullptr))))
        return hipErrorInvalidValue;
    const bool some = width > 0;
    if (any_overlap({drows != nullptr && some ? matrix(drows, n, width, lddrows) : kNone,
                     dweights != nullptr ? matrix(dweights, tokens, top, ldw) : kNone},
                    {list(position, n), some ? matrix(dout, tokens, width, lddout) : kNone,
                     dweights != nullptr && some ? matrix(rows, n, width, ldrows) : kNone,
                     weights != nullptr ? matrix(weights, tokens, top, ldw) : kNone}))
        return hipErrorInvalidValue;
    return sgemm::launch_route_combine_grad({tokens, top}, width, position, weights, ldw, rows,
                                            ldrows, dout, lddout, drows, lddrows, dweights,
                                            stream);
}

extern "C" hipError_t sgemm_f32_grouped(int transb, int rows, int N, int K, int experts,
                                        const int *offsets, float alpha, const float *A, int lda,
                                        const float *B, int ldb, long long strideb, float beta,
                                        float *C, int ldc, hipStream_t stream) {
    const bool tb = transb == SGEMM_F32_OP_T;
    if ((!tb && transb != SGEMM_F32_OP_N) || !valid_size(rows) || !valid_size(N) ||
        !valid_size(K) || !valid_size(experts) || strideb < 0 || lda < at_least_one(K) ||
        ldb < at_least_one(tb ? K : N) || ldc < at_least_one(N))
        return hipErrorInvalidValue;
    if (rows == 0 || N == 0 || experts == 0) return hipSuccess;
    if (offsets == nullptr || C == nullptr) return hipErrorInvalidValue;
    const bool product = K > 0 && alpha != 0.0f;
    if (product && (A == nullptr || B == nullptr)) return hipErrorInvalidValue;
    if (any_overlap({matrix(C, rows, N, ldc)},
                    {list(offsets, (int64_t)experts + 1),
                     product ? matrix(A, rows, K, lda) : kNone,
                     product ? sgemm::extent(B, experts, strideb, tb ? N : K, tb ? K : N, ldb, 4)
                             : kNone}))
        return hipErrorInvalidValue;
    return sgemm::launch_grouped({rows, N, K, experts, offsets, A, lda, B, ldb, strideb, C, ldc,
                                  tb, alpha, beta},
                                 stream);
}

extern "C" hipError_t sgemm_f32_grouped_ta(int rows, int M, int N, int experts,
                                           const int *offsets, float alpha, const float *A,
                                           int lda, const float *D, int ldd, float beta, float *C,
                                           int ldc, long long stridec, hipStream_t stream) {
    if (!valid_size(rows) || !valid_size(M) || !valid_size(N) || !valid_size(experts) ||
        lda < at_least_one(M) || ldd < at_least_one(N) || ldc < at_least_one(N))
        return hipErrorInvalidValue;
    if (M == 0 || N == 0 || experts == 0) return hipSuccess;
    // one C_e must not reach into the next
    if (experts > 1 && stridec < (int64_t)(M - 1) * ldc + N) return hipErrorInvalidValue;
    if (offsets == nullptr || C == nullptr) return hipErrorInvalidValue;
    const bool product = rows > 0 && alpha != 0.0f;
    if (product && (A == nullptr || D == nullptr)) return hipErrorInvalidValue;
    if (any_overlap({sgemm::extent(C, experts, experts > 1 ? stridec : 0, M, N, ldc, 4)},
                    {list(offsets, (int64_t)experts + 1),
                     product ? matrix(A, rows, M, lda) : kNone,
                     product ? matrix(D, rows, N, ldd) : kNone}))
        return hipErrorInvalidValue;
    return sgemm::launch_grouped_ta({rows, M, N, experts, offsets, A, lda, D, ldd, C, ldc,
                                     stridec, alpha, beta},
                                    stream);
}
