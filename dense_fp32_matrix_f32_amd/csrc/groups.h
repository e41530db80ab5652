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
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // lane 15 to row 1, 47 to 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
    return x;
}

// Blocks of an expert's rows, as counts of its rows: all blocks of `block` rows, the full
// ones, and the blocks of `part` rows that the rows past the full ones take.
struct AllBlocks {
    int block;
    __device__ __forceinline__ int operator()(int rows) const {
        return (int)(((int64_t)rows + block - 1) / block);
    }
};
struct FullBlocks {
    int block;
    __device__ __forceinline__ int operator()(int rows) const { return rows / block; }
};
struct RestBlocks {
    int block, part;
    __device__ __forceinline__ int operator()(int rows) const {
        return (rows % block + part - 1) / part;
    }
};

// The experts' blocks, counted expert by expert: the expert of block `item`, its first
// row and one past its last, and the block's number within the expert.  Returns false
// past the last block.  Called by every lane of a wave with the same arguments; lane l
// looks at expert base + l, 64 experts at a time.
template <class Count>
__device__ __forceinline__ bool find_expert(const int *__restrict__ offsets, int experts,
                                            int rows, const Count &count, int item, int *expert,
                                            int *first, int *end, int *index) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < experts; base += 64) {
        const int e = base + lane;
        int lo = 0, hi = 0;
        if (e < experts) {
            lo = clamp_row(offsets[e], rows);
            hi = max(lo, clamp_row(offsets[e + 1], rows));
        }
        const int mine = count(hi - lo);
        const int upto = wave_scan(mine);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        if (item < total) {
            const unsigned long long past = __ballot(upto > item);
            if (past == 0) return false;
            const int l = __builtin_ctzll(past);
            *expert = base + l;
            *first = __builtin_amdgcn_readlane(lo, l);
            *end = __builtin_amdgcn_readlane(hi, l);
            *index = item - __builtin_amdgcn_readlane(upto - mine, l);
            return *index >= 0;  // offsets that are no running sum can make the counts wrap
        }
        item -= total;
    }
    return false;
}

// How many blocks there are, for every lane of a wave.
template <class Count>
__device__ __forceinline__ int count_blocks(const int *__restrict__ offsets, int experts, int rows,
                                            const Count &count) {
    const int lane = threadIdx.x & 63;
    int all = 0;
    for (int base = 0; base < experts; base += 64) {
        const int e = base + lane;
        int mine = 0;
        if (e < experts) {
            const int lo = clamp_row(offsets[e], rows);
            mine = count(max(lo, clamp_row(offsets[e + 1], rows)) - lo);
        }
        all += __builtin_amdgcn_readlane(wave_scan(mine), 63);
    }
    return all;
}

// Block `item` of the experts' rows cut into blocks of `block`: its expert, its first row
// and one past the expert's last row.
__device__ __forceinline__ bool find_block(const int *__restrict__ offsets, int experts, int rows,
                                           int block, int item, int *expert, int *first,
                                           int *end) {
    int start, index;
    if (!find_expert(offsets, experts, rows, AllBlocks{block}, item, expert, &start, end, &index))
        return false;
    *first = start + index * block;
    return *first >= start && *first < *end;
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
