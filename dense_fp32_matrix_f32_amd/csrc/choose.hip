// choose.hip -- the experts of a token: the largest of its logits, with the weights that a
// softmax gives them, and the gradient of those weights.
//
//     w_j = exp(x[id_j] - m) / Z,  Z = sum of exp(x[e] - m) over the chosen e, or over all
//     dx[e] = sum over j with id_j = e of w_j * (dw_j - S)             (chosen)
//     dx[e] = p_e * (sum over j with id_j = e of dw_j - S)             (all; p_e = exp(x[e] - m) / Z)
//     S = sum over j of w_j * dw_j
//
// A wave takes a token.  Lane l holds V logits side by side, l V .. l V + V - 1, as integers in
// the order of the numbers, sorted largest first with the lowest number first among equal
// ones.  The largest over the lanes' first ones, in the lowest lane that has it, is the next choice,
// and that lane moves its list up.  Nothing but the logits is read and nothing but the
// results written; many tokens are bound by vector instructions (32768 tokens, 8 of 256:
// choice 23 us, gradient 20, against 7 and 14 to move the bytes; looking at all V logits in
// every round, and sums over lanes through LDS: 31 and 28; two tokens a wave, eight logits a
// lane: choice 42).  A token of 129 to 256 experts takes 47 of them for each choice, most of
// them for the steps over the lanes and for the lists, which the compiler moves up by selects over
// the whole list, 89 for its sort and about 100 for the exponentials and the sums: of 549 two
// thirds are the choices'.  Up to 512 experts a choice is 151 instructions, up to 1024 it is 647.
#include "experts.h"
#include "groups.h"

namespace sgemm {

namespace {

template <int CTRL, int ROWS>
__device__ __forceinline__ int from_lane(int x, int old) {
    return __builtin_amdgcn_update_dpp(old, x, CTRL, ROWS, 0xf, false);
}

// The largest over the lanes of a wave, for all of them.
__device__ __forceinline__ int wave_max(int x) {
    x = max(x, from_lane<0x111, 0xf>(x, x));
    x = max(x, from_lane<0x112, 0xf>(x, x));
    x = max(x, from_lane<0x114, 0xf>(x, x));
    x = max(x, from_lane<0x118, 0xf>(x, x));
    x = max(x, from_lane<0x142, 0xa>(x, x));
    x = max(x, from_lane<0x143, 0xc>(x, x));
    return __builtin_amdgcn_readlane(x, 63);
}

// The sum over the lanes of a wave, in a fixed order, for all of them.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_lane(float x) {
    return x + __builtin_bit_cast(float, from_lane<CTRL, ROWS>(__builtin_bit_cast(int, x), 0));
}
__device__ __forceinline__ float wave_sum(float x) {
    x = add_lane<0x111, 0xf>(x);
    x = add_lane<0x112, 0xf>(x);
    x = add_lane<0x114, 0xf>(x);
    x = add_lane<0x118, 0xf>(x);
    x = add_lane<0x142, 0xa>(x);
    x = add_lane<0x143, 0xc>(x);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

constexpr float kNone = -__builtin_inff();

// A logit as it counts: NaN is none, like -infinity.
__device__ __forceinline__ float logit(float x) { return x == x ? x : kNone; }

// exp(x - m), 1 for the largest itself (also where both are infinite).
__device__ __forceinline__ float term(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// The same for a sum in which the largest is 1: 2^t by the instruction, t = (x - m) log2(e)
// rounded, and what t lacks put back by its first power.  Terms below 2^-126 become zero, and
// so does that of -infinity (NaN only where m is none, whose sum is not used).
__device__ __forceinline__ float summand(float x, float m) {
    const float d = fmaxf(x - m, -200.0f), t = d * 1.44269502f;
    const float rest = fmaf(d, 1.92596299e-8f, fmaf(d, 1.44269502f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return x == m ? 1.0f : fmaf(e, rest * 0.693147182f, e);
}

// Numbers as integers in the same order (-0 as 0), and back.
__device__ __forceinline__ int key_of(float x) {
    const int b = __builtin_bit_cast(int, x + 0.0f);
    return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_key(int k) {
    return __builtin_bit_cast(float, k ^ (k >> 31 & 0x7FFFFFFF));
}
constexpr int kNoKey = (int)0x807FFFFF;  // of -infinity

// A lane's V logits from `base` on, none past the last.
template <int V>
__device__ __forceinline__ void load_logits(const float *row, int base, int experts,
                                            float (&x)[V]) {
    if (base + V <= experts) {
        __builtin_memcpy(x, __builtin_assume_aligned(row + base, 4), 4 * V);
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = logit(x[v]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = base + v < experts ? logit(row[base + v]) : kNone;
    }
}

// Largest first, the lowest place first among equal ones (Batcher's odd-even merge sort).
template <int V>
__device__ __forceinline__ void sort(int (&key)[V], int (&place)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        int &ka = key[i + j], &kb = key[i + j + k];
                        int &pa = place[i + j], &pb = place[i + j + k];
                        const bool swap = kb > ka || (kb == ka && pb < pa);
                        const int k0 = swap ? kb : ka, k1 = swap ? ka : kb;
                        const int p0 = swap ? pb : pa, p1 = swap ? pa : pb;
                        ka = k0;
                        kb = k1;
                        pa = p0;
                        pb = p1;
                    }
}

template <int V>
__global__ __launch_bounds__(256) void choose_kernel(int tokens, int experts, int top,
                                                    bool over_all, const float *logits,
                                                    int64_t ld, int *ids, float *weights) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tokens;
         t += (int64_t)gridDim.x * 4) {
        float x[V];
        load_logits<V>(logits + t * ld, lane * V, experts, x);
        int key[V], place[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = key_of(x[v]);
            place[v] = lane * V + v;
        }
        sort<V>(key, place);
        int mine = kNoKey, id = -1;  // lane j: choice j
        float most = kNone;
        for (int j = 0; j < top; ++j) {
            const int best = wave_max(key[0]);
            if (best <= kNoKey) break;
            const int from = __builtin_ctzll(__ballot(key[0] == best));
            const int won = __builtin_amdgcn_readlane(place[0], from);
            if (j == 0) most = of_key(best);
            if (lane == j) {
                mine = best;
                id = won;
            }
            const bool moves = lane == from;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) {
                key[v] = moves ? key[v + 1] : key[v];
                place[v] = moves ? place[v + 1] : place[v];
            }
            key[V - 1] = moves ? kNoKey : key[V - 1];
        }
        const float part = id >= 0 ? term(of_key(mine), most) : 0.0f;
        float z = part;
        if (over_all) {
            z = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) z += summand(x[v], most);
        }
        z = wave_sum(z);
        if (lane < top) {
            ids[t * top + lane] = id;
            weights[t * top + lane] = id >= 0 ? part / z : 0.0f;
        }
    }
}

// More experts than 16 a lane: the logits are read again for every choice, looking past
// the last one chosen.
__global__ __launch_bounds__(256) void choose_many_kernel(int tokens, int experts, int top,
                                                         bool over_all, const float *logits,
                                                         int64_t ld, int *ids, float *weights) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tokens;
         t += (int64_t)gridDim.x * 4) {
        const float *row = logits + t * ld;
        int mine = kNoKey, id = -1, before = INT32_MAX, at = -1;
        float most = kNone;
        for (int j = 0; j < top; ++j) {
            int m = kNoKey, e = INT32_MAX;
            for (int i = lane; i < experts; i += 64) {
                const int k = key_of(logit(row[i]));
                if (k > m && (k < before || (k == before && i > at))) {
                    m = k;
                    e = i;
                }
            }
            const int best = wave_max(m);
            if (best <= kNoKey) break;
            // the lowest number among equal ones
            const int won = -1 - wave_max(m == best ? -1 - e : INT32_MIN);
            if (j == 0) most = of_key(best);
            if (lane == j) {
                mine = best;
                id = won;
            }
            before = best;
            at = won;
        }
        const float part = id >= 0 ? term(of_key(mine), most) : 0.0f;
        float z = part;
        if (over_all) {
            z = 0.0f;
            for (int i = lane; i < experts; i += 64) {
                const float y = logit(row[i]);
                z += y > kNone ? term(y, most) : 0.0f;
            }
        }
        z = wave_sum(z);
        if (lane < top) {
            ids[t * top + lane] = id;
            weights[t * top + lane] = id >= 0 ? part / z : 0.0f;
        }
    }
}

// V == 0: more experts than 16 a lane, read where they are needed.
template <int V>
__global__ __launch_bounds__(256) void choose_grad_kernel(int tokens, int experts, int top,
                                                         bool over_all, const float *dweights,
                                                         const float *logits, int64_t ld,
                                                         const int *ids, const float *weights,
                                                         float *dlogits, int64_t ldd) {
    const int lane = threadIdx.x & 63;
    constexpr int HELD = V > 0 ? V : 1;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tokens;
         t += (int64_t)gridDim.x * 4) {
        int id = -1;
        float w = 0.0f, dw = 0.0f;
        if (lane < top) {
            id = ids[t * top + lane];
            if (id >= 0 && id < experts) {
                w = weights[t * top + lane];
                dw = dweights[t * top + lane];
            } else {
                id = -1;
            }
        }
        const float mean = wave_sum(w * dw);
        const float *row = logits + t * ld;
        float x[HELD], z = 0.0f;
        int most = kNoKey;
        if (over_all) {
            if constexpr (V > 0) {
                load_logits<V>(row, lane * V, experts, x);
#pragma unroll
                for (int v = 0; v < V; ++v) most = max(most, key_of(x[v]));
            } else {
                for (int e = lane; e < experts; e += 64) most = max(most, key_of(logit(row[e])));
            }
            most = wave_max(most);
            if constexpr (V > 0) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = x[v] > kNone ? term(x[v], of_key(most)) : 0.0f;
                    z += x[v];
                }
            } else {
                for (int e = lane; e < experts; e += 64) {
                    const float y = logit(row[e]);
                    z += y > kNone ? term(y, of_key(most)) : 0.0f;
                }
            }
            z = wave_sum(z);
        }
        // what a pair adds at its expert
        const float give = over_all ? dw : w * (dw - mean);
        const float inverse = z > 0.0f ? 1.0f / z : 0.0f;
        // the sums of what is given to experts e, e + 1, ...
        auto given = [&](int e, auto &sum) {
            for (int j = 0; j < top; ++j) {
                const int to = __builtin_amdgcn_readlane(id, j) - e;
                const float g = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, give), j));
#pragma unroll
                for (int v = 0; v < HELD; ++v) sum[v] += to == v ? g : 0.0f;
            }
        };
        float *out = dlogits + t * ldd;
        if constexpr (V > 0) {
            float sum[V] = {};
            given(lane * V, sum);
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] = over_all ? x[v] * inverse * (sum[v] - mean) : sum[v];
            if (lane * V + V <= experts) {
                __builtin_memcpy(__builtin_assume_aligned(out + lane * V, 4), sum, 4 * V);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (lane * V + v < experts) out[lane * V + v] = sum[v];
            }
        } else {
            for (int base = 0; base < experts; base += 64) {
                const int e = base + lane;
                float sum[1] = {};
                given(e, sum);
                const float y = over_all && e < experts ? logit(row[e]) : kNone;
                const float share = y > kNone ? term(y, of_key(most)) : 0.0f;
                if (e < experts) out[e] = over_all ? share * inverse * (sum[0] - mean) : sum[0];
            }
        }
    }
}

unsigned token_groups(int tokens) {
    const int64_t groups = ((int64_t)tokens + 3) / 4;
    return (unsigned)(groups < most_groups(256) ? groups : most_groups(256));
}

}  // namespace

hipError_t launch_route_choose(int tokens, int experts, int top, bool over_all, const float *logits,
                               int64_t ld, int *ids, float *weights, hipStream_t s) {
    const dim3 grid(token_groups(tokens)), block(256);
    auto run = [&](auto kernel) {
        return launch(kernel, grid, block, 0, s, tokens, experts, top, over_all, logits, ld, ids,
                      weights);
    };
    if (experts <= 64) return run(choose_kernel<1>);
    if (experts <= 128) return run(choose_kernel<2>);
    if (experts <= 256) return run(choose_kernel<4>);
    if (experts <= 512) return run(choose_kernel<8>);
    if (experts <= 1024) return run(choose_kernel<16>);
    return run(choose_many_kernel);
}

hipError_t launch_route_choose_grad(int tokens, int experts, int top, bool over_all,
                                    const float *dweights, const float *logits, int64_t ld,
                                    const int *ids, const float *weights, float *dlogits,
                                    int64_t ldd, hipStream_t s) {
    const dim3 grid(token_groups(tokens)), block(256);
    auto run = [&](auto kernel) {
        return launch(kernel, grid, block, 0, s, tokens, experts, top, over_all, dweights, logits,
                      ld, ids, weights, dlogits, ldd);
    };
    if (experts <= 64) return run(choose_grad_kernel<1>);
    if (experts <= 128) return run(choose_grad_kernel<2>);
    if (experts <= 256) return run(choose_grad_kernel<4>);
    if (experts <= 512) return run(choose_grad_kernel<8>);
    if (experts <= 1024) return run(choose_grad_kernel<16>);
    return run(choose_grad_kernel<0>);
}

}  // namespace sgemm
