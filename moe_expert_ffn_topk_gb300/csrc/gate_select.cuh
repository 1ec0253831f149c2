// The router's selection, one warp per token: scores, groups, top-k and weights (see moe_gate in moe_ops.h).
#pragma once

#include "common.cuh"
#include "ops.h"

namespace moe {

// Order of fp32 values as unsigned integers: a > b exactly when key(a) > key(b). -0 and +0 get the same key (they
// compare equal, so the index decides between them); 0 is below every key of a number and marks "not available".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// s = 1 / (1 + e^-l) in fp32, rounded to nearest in the last step (the selection compares these values, so the fast exp and divide
// of the activations are not used here). The reciprocal is an estimate and two Newton steps with fused multiply-adds, without the
// branch of a division: a lane's scores then overlap (8 of them: 2450 cycles with divisions, one after another). Above 2^120 the
// divisor is taken down by 2^64 and the result with it, as the steps would leave the range.
__device__ __forceinline__ float gate_sigmoid(float l) {
    const float x = __fadd_rn(1.0f, expf(-l));
    const float scale = x >= 1.329228e36f ? 5.4210109e-20f : 1.0f, d = x * scale;  // 2^120, 2^-64
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = __fmaf_rn(__fmaf_rn(-d, r, 1.0f), r, r);
    r = __fmaf_rn(__fmaf_rn(-d, r, 1.0f), r, r);
    return x <= 3.4028235e38f ? r * scale : x == x ? 0.0f : x;
}

// Floats of shared memory that gate_token works in, per warp: logits, bias, choice keys (a few words apart per group,
// see there), selected ids.
__host__ __device__ inline int gate_scratch(int E) { return 3 * E + 64; }

// One token, by one warp. scratch: gate_scratch(E) words of shared memory of this warp, the first E holding the logits, the
// next E the bias where there is one (this function separates its reads from their writes). Selected experts go to ids[0..K) and weights[0..K).
//
// Rows stay in shared memory, not in registers, and every loop is kept rolled: few tokens run this once, and then what counts
// is how much code has to be fetched (7 tokens, 256 experts, on the device: 6.9 us with the row in registers and everything
// unrolled, 6.3 when first rolled, 5.1 now).
__device__ __forceinline__ void gate_token(float* scratch, bool has_bias, const moe_gate_options& o, int E, int K, int lane,
                                           int32_t* ids, float* weights) {
    constexpr uint32_t kAll = 0xffffffffu;
    const float *logit = scratch, *bias = scratch + E;
    uint32_t* key = reinterpret_cast<uint32_t*>(scratch + 2 * E);
    int* chosen = reinterpret_cast<int*>(scratch + 3 * E + 32);
    const bool softmax = o.score == MOE_SCORE_SOFTMAX;
    const bool groups = o.num_groups > 1;
    // group of expert e: (e + 0.5) / size truncated, exact for e < 1024; `per` lanes scan a group, and keys of a group are `per`
    // words further on than those of the one before, which keeps the lanes' banks apart
    const int size = E / o.num_groups;
    const float inv_size = __fdividef(1.0f, (float)size);
    int per = 32;
    while (per * o.num_groups > 32) per >>= 1;
    const int pad = groups ? per : 0;
    auto group_of = [&](int e) { return (int)(((float)e + 0.5f) * inv_size); };
    __syncwarp();

    float top = -INFINITY, total = 1.0f;
    if (softmax) {
#pragma unroll 4
        for (int e = lane; e < E; e += 32) top = fmaxf(top, logit[e]);  // fmaxf passes over NaNs
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    }
    const bool inf = top == INFINITY;
    auto exp_of = [&](float l) { return inf ? (l == INFINITY ? 1.0f : 0.0f) : expf(l - top); };
    if (softmax) {
        float sum = 0.0f;
#pragma unroll 2
        for (int e = lane; e < E; e += 32) {
            const float l = logit[e];
            sum += l > -INFINITY ? exp_of(l) : 0.0f;
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        total = sum;
    }
    auto score = [&](float l) { return softmax ? __fdiv_rn(exp_of(l), total) : gate_sigmoid(l); };

    // choice keys: 0 = not available. A loop for each kind of score, four experts at a time and read before the first is
    // written: their chains of some 250 cycles overlap.
    auto make_keys = [&](auto value) {
        for (int e = lane; e < E; e += 128) {
            float l[4], c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                l[j] = e + 32 * j < E ? logit[e + 32 * j] : -INFINITY;
                c[j] = has_bias && e + 32 * j < E ? bias[e + 32 * j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] += value(l[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + 32 * j < E)  // not for a NaN either
                    key[e + 32 * j + group_of(e + 32 * j) * pad] = l[j] > -INFINITY && c[j] == c[j] ? order_key(c[j]) : 0u;
        }
    };
    if (!softmax) make_keys([](float l) { return gate_sigmoid(l); });
    else if (has_bias) make_keys(score);
    else make_keys([](float l) { return l; });

    uint32_t kept = ~0u;  // bit g: the experts of group g are eligible
    if (groups) {
        __syncwarp();
        const int g = lane / per, sub = lane & (per - 1);
        uint32_t a = 0u, b = 0u;  // keys of the group's two largest, a >= b; 0: it has no such candidate
        if (g < o.num_groups) {
#pragma unroll 4
            for (int j = sub; j < size; j += per) {
                const uint32_t k = key[g * (size + pad) + j];
                b = max(b, min(a, k));
                a = max(a, k);
            }
        }
        for (int d = 1; d < per; d <<= 1) {
            const uint32_t a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
            b = max(min(a, a2), max(b, b2));
            a = max(a, a2);
        }
        // the sum over the candidates there are; 0, below the rank of any group with one, without (+inf is a rank of its own: what
        // the second adds to it does not count)
        uint32_t rank = 0u;
        if (a != 0u && sub == 0) {
            const float first = key_value(a);
            rank = order_key(o.group_top == 2 && b != 0u && first < INFINITY ? first + key_value(b) : first);
        }
        kept = 0u;  // (a bit more does no harm where only groups without a candidate are left)
        for (int k = 0; k < o.topk_groups; ++k) {
            const uint32_t best = __reduce_max_sync(kAll, rank);
            const int win = __ffs(__ballot_sync(kAll, rank == best)) - 1;  // the lowest lane: the lowest group
            kept |= 1u << __shfl_sync(kAll, g, win);
            if (lane == win) rank = 0u;
        }
    }

    // K rounds of "largest key, lowest index"; lane k keeps the k-th. Each lane knows the best two of its own experts that are
    // left, and looks for them again only when both have been taken.
    uint32_t best1, best2;
    int at1, at2;
    auto own_best = [&]() {
        best1 = best2 = 0u;
        at1 = at2 = 0;
#pragma unroll 4
        for (int e = lane; e < E; e += 32) {
            const int h = groups ? group_of(e) : 0;
            const uint32_t c = key[e + h * pad], k = (kept >> h) & 1u ? c : 0u;
            if (k > best1) {
                best2 = best1, at2 = at1;
                best1 = k, at1 = e;
            } else if (k > best2) {
                best2 = k, at2 = e;
            }
        }
    };
    own_best();
    bool two = true;  // the second one is known
    int found = 0;
    for (; found < K; ++found) {
        const uint32_t best = __reduce_max_sync(kAll, best1);
        if (best == 0u) break;
        // one lane has it, or more (equal values): the one with the lowest index
        const uint32_t with = __ballot_sync(kAll, best1 == best);
        bool mine = best1 == best;
        if (with & (with - 1u)) mine = __reduce_min_sync(kAll, mine ? (uint32_t)at1 : 0xffffffffu) == (uint32_t)at1 && mine;
        if (mine) {
            chosen[found] = at1;
            key[at1 + (groups ? group_of(at1) : 0) * pad] = 0u;
            if (two) {
                best1 = best2, at1 = at2;
            } else {
                own_best();
            }
            two = !two;
        }
        __syncwarp();
    }
    const int my_id = lane < found ? chosen[lane] : -1;
    float w = my_id >= 0 ? score(logit[my_id]) : 0.0f;
    if (o.normalize) {
        float sum = w;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        w = __fdiv_rn(w, sum + 1e-20f);
    }
    w *= o.route_scale;
    if (lane < K) {
        ids[lane] = my_id;
        weights[lane] = my_id >= 0 ? w : 0.0f;
    }
}

}  // namespace moe
