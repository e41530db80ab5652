// groups.h -- rows that belong to experts: expert e owns rows offsets[e] ..
// offsets[e+1]-1 of an array of `rows` rows, offsets on the device.
#pragma once

#include "internal.h"

namespace sgemm {

// First row of the range that starts at offsets[e], and one past the last of the
// range that ends at offsets[e+1], whatever the array holds: clamped to the rows.
__device__ __forceinline__ int clamp_row(int x, int rows) { return max(0, min(x, rows)); }

// Inclusive sum over the lanes of a wave, in six additions (data-parallel moves
// within rows of 16 lanes, then the rows' last lanes broadcast to the next rows).
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);  // from 1 lane before
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);  // 2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);  // 4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);  // 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // lane 15 to row 1, 47 to row 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
    return x;
}

// The experts' rows cut into blocks of `block`, counted expert by expert: the
// expert of block `item`, its first row and one past the expert's last row.
// Returns false past the last block.  Called by every lane of a wave with the
// same arguments; lane l looks at expert base + l, 64 experts at a time.
__device__ __forceinline__ bool find_block(const int *__restrict__ offsets, int experts, int rows,
                                           int block, int item, int *expert, int *first,
                                           int *end) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < experts; base += 64) {
        const int e = base + lane;
        int lo = 0, hi = 0;
        if (e < experts) {
            lo = clamp_row(offsets[e], rows);
            hi = max(lo, clamp_row(offsets[e + 1], rows));
        }
        const int mine = (int)(((int64_t)hi - lo + block - 1) / block);
        const int upto = wave_scan(mine);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        if (item < total) {
            const unsigned long long past = __ballot(upto > item);
            if (past == 0) return false;
            const int l = __builtin_ctzll(past);
            const int start = __builtin_amdgcn_readlane(lo, l);
            *expert = base + l;
            *end = __builtin_amdgcn_readlane(hi, l);
            *first = start + (item - __builtin_amdgcn_readlane(upto - mine, l)) * block;
            // offsets that are no running sum can make the counts wrap
            return *first >= start && *first < *end;
        }
        item -= total;
    }
    return false;
}

// How many blocks there are, for every lane of a wave.
__device__ __forceinline__ int count_blocks(const int *__restrict__ offsets, int experts, int rows,
                                            int block) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int base = 0; base < experts; base += 64) {
        const int e = base + lane;
        int mine = 0;
        if (e < experts) {
            const int lo = clamp_row(offsets[e], rows);
            const int hi = max(lo, clamp_row(offsets[e + 1], rows));
            mine = (int)(((int64_t)hi - lo + block - 1) / block);
        }
        count += __builtin_amdgcn_readlane(wave_scan(mine), 63);
    }
    return count;
}

// The most work-groups of `threads` work-items that one launch holds: its work-items
// are counted in 32 bits.
constexpr int64_t most_groups(int threads) { return UINT32_MAX / threads; }

// The most blocks find_block() can find: each expert with rows ends at most one
// block short of full.
inline int64_t most_blocks(int rows, int experts, int block) {
    const int64_t with_rows = rows < experts ? rows : experts;
    return (rows - with_rows) / block + with_rows;
}

}  // namespace sgemm
