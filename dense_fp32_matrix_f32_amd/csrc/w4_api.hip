// w4_api.hip -- the entry points of include/sgemm_f32_w4.h: argument validation on
// the host (before any HIP call) and launch on the caller's stream.
#include "sgemm_f32_w4.h"

#include "extent.h"
#include "w4.h"

using sgemm::Extent;
using sgemm::valid_size;
using sgemm::W4Layout;

namespace {

int at_least_one(int x) { return x > 1 ? x : 1; }

bool valid_format(int experts, int N, int K, int group, int scale_type) {
    return valid_size(experts) && valid_size(N) && valid_size(K) && group > 0 &&
           (group == 32 || group == 64 || group % sgemm::kW4Block == 0) &&
           scale_type >= SGEMM_F32_W4_SCALE_F32 && scale_type <= SGEMM_F32_W4_SCALE_BF16;
}

// Bytes of the packed array, or -1 where they pass 62 bits.
int64_t packed_bytes_of(const W4Layout &l, int experts) {
    const __int128 bytes = (__int128)l.strips * l.blocks * l.record * experts;
    return bytes > ((__int128)1 << 62) ? -1 : (int64_t)bytes;
}

// The packed array of a call: present, aligned, large enough.
bool valid_packed(const W4Layout &l, int experts, const void *packed, size_t bytes) {
    const int64_t need = packed_bytes_of(l, experts);
    return need >= 0 && packed != nullptr && ((uintptr_t)packed & 15) == 0 &&
           bytes >= (size_t)need;
}

Extent packed_extent(const W4Layout &l, int experts, const void *packed) {
    return sgemm::bytes_from(packed, packed_bytes_of(l, experts));
}

hipError_t product(int rows, int N, int K, int experts, const int *offsets, const float *A, int lda,
                   const void *packed, int group, int scale_type, int zeros, float *C, int ldc,
                   hipStream_t stream) {
    const W4Layout l = sgemm::w4_layout(N, K, group, scale_type, zeros);
    const Extent c = sgemm::extent(C, rows, N, ldc, 4);
    if (K > 0) {
        if (A == nullptr || !valid_packed(l, experts, packed, SIZE_MAX))
            return hipErrorInvalidValue;
        if (sgemm::overlaps(c, sgemm::extent(A, rows, K, lda, 4)) ||
            sgemm::overlaps(c, packed_extent(l, experts, packed)))
            return hipErrorInvalidValue;
    }
    if (offsets != nullptr &&
        sgemm::overlaps(c, sgemm::extent(offsets, 1, (int64_t)experts + 1, 1, 4)))
        return hipErrorInvalidValue;
    return sgemm::launch_w4(
        l, {rows, A, lda, (const unsigned char *)packed, C, ldc, experts, offsets}, stream);
}

}  // namespace

extern "C" size_t sgemm_f32_w4_packed_size(int experts, int N, int K, int group, int scale_type,
                                           int zeros) {
    if (!valid_format(experts, N, K, group, scale_type)) return 0;
    const W4Layout l = sgemm::w4_layout(N, K, group, scale_type, zeros);
    const int64_t bytes = packed_bytes_of(l, experts);
    return bytes < 0 ? 0 : (size_t)bytes;
}

extern "C" hipError_t sgemm_f32_w4_pack(int experts, int N, int K, int group,
                                        const unsigned char *codes, const void *scales,
                                        int scale_type, const unsigned char *zeros, void *packed,
                                        size_t packed_bytes, hipStream_t stream) {
    if (!valid_format(experts, N, K, group, scale_type)) return hipErrorInvalidValue;
    if (experts == 0 || N == 0 || K == 0) return hipSuccess;
    const W4Layout l = sgemm::w4_layout(N, K, group, scale_type, zeros != nullptr);
    if (codes == nullptr || scales == nullptr || !valid_packed(l, experts, packed, packed_bytes) ||
        ((uintptr_t)scales & (l.scale_size - 1)) != 0)
        return hipErrorInvalidValue;
    const int64_t groups = ((int64_t)K + group - 1) / group, pairs = ((int64_t)K + 1) / 2;
    const Extent out = packed_extent(l, experts, packed);
    if (sgemm::overlaps(out, sgemm::extent(codes, experts * pairs, N, N, 1)) ||
        sgemm::overlaps(out, sgemm::extent(scales, experts * groups, N, N, l.scale_size)) ||
        (zeros != nullptr && sgemm::overlaps(out, sgemm::extent(zeros, experts * groups, N, N, 1))))
        return hipErrorInvalidValue;
    return sgemm::launch_w4_pack(l, experts, codes, (const unsigned char *)scales, zeros,
                                 (unsigned char *)packed, stream);
}

extern "C" hipError_t sgemm_f32_w4_quantize(int experts, int N, int K, int group, const float *B,
                                            int ldb, long long strideb, int scale_type, int zeros,
                                            void *packed, size_t packed_bytes,
                                            hipStream_t stream) {
    if (!valid_format(experts, N, K, group, scale_type) || ldb < at_least_one(N) ||
        strideb < 0)
        return hipErrorInvalidValue;
    if (experts == 0 || N == 0 || K == 0) return hipSuccess;
    const W4Layout l = sgemm::w4_layout(N, K, group, scale_type, zeros);
    if (B == nullptr || !valid_packed(l, experts, packed, packed_bytes) ||
        sgemm::overlaps(packed_extent(l, experts, packed),
                        sgemm::extent(B, experts, strideb, K, N, ldb, 4)))
        return hipErrorInvalidValue;
    return sgemm::launch_w4_quantize(l, experts, B, ldb, strideb, (unsigned char *)packed, stream);
}

extern "C" hipError_t sgemm_f32_w4_unpack(int experts, int N, int K, int group, int scale_type,
                                          int zeros, const void *packed, size_t packed_bytes,
                                          float *B, int ldb, long long strideb,
                                          hipStream_t stream) {
    if (!valid_format(experts, N, K, group, scale_type) || ldb < at_least_one(N))
        return hipErrorInvalidValue;
    if (experts == 0 || N == 0 || K == 0) return hipSuccess;
    // one matrix must not reach into the next
    if (experts > 1 && strideb < (int64_t)(K - 1) * ldb + N) return hipErrorInvalidValue;
    const W4Layout l = sgemm::w4_layout(N, K, group, scale_type, zeros);
    if (B == nullptr || !valid_packed(l, experts, packed, packed_bytes) ||
        sgemm::overlaps(packed_extent(l, experts, packed),
                        sgemm::extent(B, experts, experts > 1 ? strideb : 0, K, N, ldb, 4)))
        return hipErrorInvalidValue;
    return sgemm::launch_w4_unpack(l, experts, (const unsigned char *)packed, B, ldb, strideb,
                                   stream);
}

extern "C" hipError_t sgemm_f32_w4(int M, int N, int K, const float *A, int lda,
                                   const void *packed, int group, int scale_type, int zeros,
                                   float *C, int ldc, hipStream_t stream) {
    if (!valid_size(M) || !valid_format(1, N, K, group, scale_type) || lda < at_least_one(K) ||
        ldc < at_least_one(N))
        return hipErrorInvalidValue;
    if (M == 0 || N == 0) return hipSuccess;
    if (C == nullptr) return hipErrorInvalidValue;
    return product(M, N, K, 1, nullptr, A, lda, packed, group, scale_type, zeros, C, ldc, stream);
}

extern "C" hipError_t sgemm_f32_w4_experts(int rows, int N, int K, int experts, const int *offsets,
                                           const float *A, int lda, const void *packed, int group,
                                           int scale_type, int zeros, float *C, int ldc,
                                           hipStream_t stream) {
    if (!valid_size(rows) || !valid_format(experts, N, K, group, scale_type) ||
        lda < at_least_one(K) || ldc < at_least_one(N))
        return hipErrorInvalidValue;
    if (rows == 0 || N == 0 || experts == 0) return hipSuccess;
    if (C == nullptr || offsets == nullptr) return hipErrorInvalidValue;
    return product(rows, N, K, experts, offsets, A, lda, packed, group, scale_type, zeros, C, ldc,
                   stream);
}
