// f8_pack.hip -- numbers into 8-bit floating point with a scale for each block of 128, and
// weights from codes and back (layout in f8.h).  Each number is read once and each code written
// once, and what bounds it is moving them: 8192 x 8192 from fp32 67 us, with the transpose 82,
// from codes 36 (transposed codes 25), back to fp32 97, which is 5.0, 4.9, 3.7 (5.5) and 3.5
// TB/s next to 5.1 of a copy of 1 GiB; 4096 x 4096 18, 20, 15 (11) and 16 us a call.
#include "f8.h"
#include "groups.h"

namespace sgemm {

namespace {

// A work-group puts 8 rows by 4 blocks of 128 k into 8 bits, a wave one block: eight lanes a
// row, each one chunk of 16 k, so a wave reads 512 bytes of each row and writes 1024 side by
// side, and the four waves fill the rows' words of scales.
template <class T, int TYPE>
__global__ __launch_bounds__(256) void f8_rows_kernel(F8RowsProblem p, int blocks) {
    const int lane = threadIdx.x & 63, chunk = lane & 7;
    unsigned char *scales = p.q + (int64_t)blocks * p.rows * kF8Block;
    const int64_t eights = ((int64_t)p.rows + 7) / 8, items = eights * ((blocks + 3) / 4);
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int quad = (int)(item / eights), row = (int)(item % eights) * 8 + (lane >> 3);
        const int block = 4 * quad + (threadIdx.x >> 6);
        if (row >= p.rows) continue;
        unsigned char *word = scales + ((int64_t)quad * p.rows + row) * 4 + (block & 3);
        if (block >= blocks) {
            if (chunk == 0) *word = 127;
            continue;
        }
        const int k = block * kF8Block + chunk * 16;
        float v[16];
        f8_load16((const T *)p.A + row * p.lda + k, p.K - k, v);
        unsigned byte;
        const uint4 out = f8_chunk<TYPE>(v, &byte);
        *(uint4 *)(p.q + ((int64_t)block * p.rows + row) * kF8Block + f8_place(chunk, row)) = out;
        if (chunk == 0) *word = (unsigned char)byte;
    }
}

// A work-group puts 64 columns of one block of 128 rows into 8 bits: a wave 32 of the rows, a
// lane one column, with 256 bytes of each row read side by side.
template <class T, int TYPE>
__global__ __launch_bounds__(256) void f8_columns_kernel(F8ColumnsProblem p) {
    __shared__ float part[4][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned char *scales = p.q + p.blocks * p.width * kF8Block;
    const int64_t strips = ((int64_t)p.width + 63) / 64;
    for (int64_t item = blockIdx.x; item < p.blocks * strips; item += gridDim.x) {
        const int64_t block = item / strips;
        const int col = (int)(item % strips) * 64 + lane;
        int e = 0, first = (int)block * kF8Block, end = p.rows;
        if (p.offsets != nullptr &&
            !find_block(p.offsets, p.experts, p.rows, kF8Block, (int)block, &e, &first, &end))
            return;  // (later items are of this block or further ones)
        const int row0 = first + 32 * wave, left = end - row0;
        float v[32];
        float most = 0.0f;
        const T *x = (const T *)p.A + (int64_t)row0 * p.lda + col;
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            v[r] = r < left && col < p.width ? (float)x[r * p.lda] : 0.0f;
            most = fmaxf(most, f8_size(v[r]));
        }
        part[wave][lane] = most;
        __syncthreads();
        most = fmaxf(fmaxf(part[0][lane], part[1][lane]), fmaxf(part[2][lane], part[3][lane]));
        const int byte = f8_scale_byte(most, TYPE);
        const float inv = f8_inverse(byte);
        if (col < p.width) {
            unsigned char *to = p.q + (block * p.width + col) * kF8Block;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 out;
                const float *w = v + 16 * h;
                out.x = f8_codes<TYPE>(w[0], w[1], w[2], w[3], inv);
                out.y = f8_codes<TYPE>(w[4], w[5], w[6], w[7], inv);
                out.z = f8_codes<TYPE>(w[8], w[9], w[10], w[11], inv);
                out.w = f8_codes<TYPE>(w[12], w[13], w[14], w[15], inv);
                *(uint4 *)(to + f8_place(2 * wave + h, col)) = out;
            }
            if (wave == 0) scales[(block / 4 * p.width + col) * 4 + block % 4] = (unsigned char)byte;
        }
        __syncthreads();  // part[] is written again
    }
}

// A work-group forms one 128 x 128 of R x C numbers: its codes go to LDS, and from there to
// the planes along the rows as they are and to those down the columns byte by byte.
// CODES: they are given, with their scales.
template <bool CODES>
__global__ __launch_bounds__(256) void f8_matrix_kernel(F8MatrixProblem p, F8Weights down,
                                                        F8Weights along) {
    constexpr int PITCH = 132;  // bytes of a row of codes: columns meet different banks
    __shared__ __attribute__((aligned(16))) unsigned char codes[128 * PITCH];
    __shared__ float parts[4];
    const int tid = threadIdx.x;
    const int blocks_c = (int)down.cols;  // down: rows are columns
    const int64_t id = blockIdx.x;
    const int bc = (int)(id % blocks_c);
    const int br = (int)(id / blocks_c % along.cols);
    const int e = (int)(id / blocks_c / along.cols);
    const int r0 = br * kF8Block, c0 = bc * kF8Block;
    const int c = c0 + 4 * (tid & 31);
    float scale;
    if constexpr (CODES) {
        const unsigned char *src = (const unsigned char *)p.source + e * p.stride;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + (tid >> 5) + 8 * i;
            unsigned word = 0;
            if (r < p.R) {
                const unsigned char *from = src + r * p.ld + c;
                if (c + 4 <= p.C) {
                    __builtin_memcpy(&word, from, 4);
                } else {
                    for (int q = 0; q < 4; ++q)
                        if (c + q < p.C) word |= (unsigned)from[q] << (8 * q);
                }
            }
            *(unsigned *)(codes + (r - r0) * PITCH + (c - c0)) = word;
        }
        const int64_t at = ((int64_t)e * along.cols + br) * blocks_c + bc;
        if (p.scale_type == F8_SCALE_E8M0) {
            const unsigned b = ((const unsigned char *)p.scales)[at];
            // 2^-127 is half the smallest normal number, 255 is NaN
            scale = __builtin_bit_cast(float, b == 0 ? 0x400000u : b == 255 ? 0x7FC00000u : b << 23);
        } else {
            scale = ((const float *)p.scales)[at];
        }
    } else {
        const float *src = (const float *)p.source + e * p.stride;
        float v[16][4];
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + (tid >> 5) + 8 * i;
            const float *from = src + r * p.ld + c;
            if (r < p.R && c + 4 <= p.C) {
                __builtin_memcpy(v[i], from, 16);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i][q] = r < p.R && c + q < p.C ? from[q] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) most = fmaxf(most, f8_size(v[i][q]));
        }
        for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
        if ((tid & 63) == 0) parts[tid >> 6] = most;
        __syncthreads();
        most = fmaxf(fmaxf(parts[0], parts[1]), fmaxf(parts[2], parts[3]));
        const int byte = f8_scale_byte(most, F8_E4M3);
        const float inv = f8_inverse(byte);
        scale = f8_exp2(byte);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *(unsigned *)(codes + ((tid >> 5) + 8 * i) * PITCH + (c - c0)) =
                f8_codes<F8_E4M3>(v[i][0], v[i][1], v[i][2], v[i][3], inv);
    }
    __syncthreads();
    if (p.along != nullptr) {
        // 1024 chunks of 16 bytes: row r, chunk of its 128 columns (rows padded to 16 too)
        unsigned char *out = p.along + e * along.bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i, chunk = tid & 7;
            if (r0 + r < along.rows) {
                uint4 x;
                __builtin_memcpy(&x, __builtin_assume_aligned(codes + r * PITCH + 16 * chunk, 4), 16);
                *(uint4 *)(out + (bc * along.rows + r0 + r) * kF8Block + f8_place(chunk, r)) = x;
            }
        }
        if (tid == 0) ((float *)(out + along.planes))[bc * along.cols + br] = scale;
    }
    if (p.down != nullptr) {
        unsigned char *out = p.down + e * down.bytes;
        // a lane takes column n = tid % 128 and every other chunk of its 128 rows
        const int n = tid & 127;
        if (c0 + n < down.rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int chunk = 2 * i + (tid >> 7);
                unsigned w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    w[q] = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        w[q] |= (unsigned)codes[(16 * chunk + 4 * q + b) * PITCH + n] << (8 * b);
                }
                *(uint4 *)(out + (br * down.rows + c0 + n) * kF8Block + f8_place(chunk, n)) =
                    uint4{w[0], w[1], w[2], w[3]};
            }
        }
        if (tid == 0) ((float *)(out + down.planes))[br * down.cols + bc] = scale;
    }
}

// A work-item forms the 16 numbers of one chunk: consecutive k of one column.
__global__ __launch_bounds__(256) void f8_unpack_kernel(int experts, int N, int K, F8Weights l,
                                                        const unsigned char *array, float *B,
                                                        int64_t ldb, int64_t strideb) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    const int64_t chunks = ((int64_t)K + 15) / 16;
    for (int64_t item = blockIdx.y; item < chunks * experts; item += gridDim.y) {
        const int64_t e = item / chunks, chunk = item % chunks, block = chunk / 8;
        const unsigned char *packed = array + e * l.bytes;
        const uint4 x = *(const uint4 *)(packed + (block * l.rows + n) * kF8Block +
                                         f8_place((int)(chunk % 8), n));
        const float s = ((const float *)(packed + l.planes))[block * l.cols + n / kF8Block];
        const unsigned w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v[4] = {__builtin_amdgcn_cvt_f32_fp8(w[q], 0),
                                __builtin_amdgcn_cvt_f32_fp8(w[q], 1),
                                __builtin_amdgcn_cvt_f32_fp8(w[q], 2),
                                __builtin_amdgcn_cvt_f32_fp8(w[q], 3)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int64_t k = chunk * 16 + 4 * q + b;
                if (k < K) B[e * strideb + k * ldb + n] = s * v[b];
            }
        }
    }
}

template <class T>
hipError_t launch_rows_as(const F8RowsProblem &p, hipStream_t s) {
    const int64_t blocks = f8_blocks(p.K), items = ((int64_t)p.rows + 7) / 8 * ((blocks + 3) / 4);
    const dim3 grid((unsigned)(items < most_groups(256) ? items : most_groups(256)));
    return p.type == F8_E4M3
               ? launch(f8_rows_kernel<T, F8_E4M3>, grid, dim3(256), 0, s, p, (int)blocks)
               : launch(f8_rows_kernel<T, F8_E5M2>, grid, dim3(256), 0, s, p, (int)blocks);
}

template <class T>
hipError_t launch_columns_as(const F8ColumnsProblem &p, hipStream_t s) {
    const int64_t items = ((int64_t)p.width + 63) / 64 * p.blocks;
    const dim3 grid((unsigned)(items < most_groups(256) ? items : most_groups(256)));
    return p.type == F8_E4M3 ? launch(f8_columns_kernel<T, F8_E4M3>, grid, dim3(256), 0, s, p)
                             : launch(f8_columns_kernel<T, F8_E5M2>, grid, dim3(256), 0, s, p);
}

template <bool CODES>
hipError_t launch_matrix(const F8MatrixProblem &p, hipStream_t s) {
    const F8Weights down = f8_weights(p.C, p.R), along = f8_weights(p.R, p.C);
    const __int128 groups = (__int128)down.cols * along.cols * p.experts;
    if (groups > most_groups(256)) return hipErrorInvalidValue;
    return launch(f8_matrix_kernel<CODES>, dim3((unsigned)groups), dim3(256), 0, s, p, down, along);
}

}  // namespace

hipError_t launch_f8_rows(const F8RowsProblem &p, hipStream_t s) {
    return p.in == F8_IN_F32 ? launch_rows_as<float>(p, s) : launch_rows_as<Bf16>(p, s);
}

hipError_t launch_f8_columns(const F8ColumnsProblem &p, hipStream_t s) {
    return p.in == F8_IN_F32 ? launch_columns_as<float>(p, s) : launch_columns_as<Bf16>(p, s);
}

hipError_t launch_f8_quantize(const F8MatrixProblem &p, hipStream_t s) {
    return launch_matrix<false>(p, s);
}

hipError_t launch_f8_pack(const F8MatrixProblem &p, hipStream_t s) {
    return launch_matrix<true>(p, s);
}

hipError_t launch_f8_unpack(int experts, int N, int K, const unsigned char *packed, float *B,
                            int64_t ldb, int64_t strideb, hipStream_t s) {
    const int64_t items = ((int64_t)K + 15) / 16 * experts, cols = ((int64_t)N + 255) / 256;
    const dim3 grid((unsigned)cols, (unsigned)(items < 65535 ? items : 65535));
    return launch(f8_unpack_kernel, grid, dim3(256), 0, s, experts, N, K, f8_weights(N, K), packed,
                  B, ldb, strideb);
}

}  // namespace sgemm
