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

// s = 1 / (1 + e^-l) in fp32 with IEEE operations (the selection compares these values, so the fast exp and
// divide of the activations are not used here)
__device__ __forceinline__ float gate_sigmoid(float l) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l))); }

// One token. v: this lane's logits, expert i * 32 + lane in v[i], -inf where masked or past E. Selected experts go to
// ids[0..K) and weights[0..K). scratch: E + 32 floats of shared memory of this warp (groups > 1 only).
template <int kV>
__device__ __forceinline__ void gate_token(float (&v)[kV], const float* bias, const moe_gate_options& o, int E, int K,
                                           float* scratch, int lane, int32_t* ids, float* weights) {
    constexpr uint32_t kAll = 0xffffffffu;
    const bool softmax = o.score == MOE_SCORE_SOFTMAX;
    float top = -INFINITY, total = 1.0f;
    bool inf = false;
    if (softmax) {
#pragma unroll
        for (int i = 0; i < kV; ++i) top = fmaxf(top, v[i]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
        inf = top == INFINITY;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            sum += inf ? (v[i] == INFINITY ? 1.0f : 0.0f) : v[i] == -INFINITY ? 0.0f : expf(v[i] - top);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        total = sum;
    }
    auto score = [&](float l) {
        if (!softmax) return gate_sigmoid(l);
        return __fdiv_rn(inf ? (l == INFINITY ? 1.0f : 0.0f) : expf(l - top), total);
    };

    // choice keys: 0 = not available
    uint32_t key[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int e = i * 32 + lane;
        float c = v[i];
        const bool on = e < E && c > -INFINITY;  // false for a NaN too
        if (on && (bias || !softmax)) {
            c = score(c);
            if (bias) c += __ldg(bias + e);
        }
        key[i] = on && c == c ? order_key(c) : 0u;
    }

    if (o.num_groups > 1) {
        // every group is scanned by `per` lanes; padding by `per` floats a group keeps their banks apart
        const int G = o.num_groups, size = E / G;
        int per = 1;
        while (per * 2 * G <= 32) per *= 2;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int e = i * 32 + lane;
            if (e < E) scratch[e + e / size * per] = key[i] ? key_value(key[i]) : -INFINITY;
        }
        __syncwarp();
        const int g = lane / per, sub = lane % per;
        float a = -INFINITY, b = -INFINITY;  // the two largest, a >= b
        if (g < G) {
            const int first = g * (size + per);
            for (int j = sub; j < size; j += per) {
                const float c = scratch[first + j];
                b = fmaxf(b, fminf(a, c));
                a = fmaxf(a, c);
            }
        }
        for (int d = 1; d < per; d <<= 1) {
            const float a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        }
        const float rank = o.group_top == 1 || size == 1 ? a : a + b;
        uint32_t rk = g < G && sub == 0 ? order_key(rank) : 0u;  // of -inf too: a fully masked group still has a rank
        uint32_t kept = 0;                                       // bit g
        for (int k = 0; k < o.topk_groups; ++k) {
            const uint32_t best = __reduce_max_sync(kAll, rk);
            const int win = __ffs(__ballot_sync(kAll, rk == best)) - 1;  // the lowest lane: the lowest group
            kept |= 1u << (win / per);
            if (lane == win) rk = 0u;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int e = i * 32 + lane;
            if (e < E && !((kept >> (e / size)) & 1u)) key[i] = 0u;
        }
    }

    // K rounds of "largest key, lowest index"; lane k keeps the k-th
    uint32_t mine = 0;
    int at = 0;
    auto local_best = [&]() {
        mine = 0;
        at = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (key[i] > mine) {
                mine = key[i];
                at = i;
            }
    };
    local_best();
    int my_id = -1;
    float my_logit = 0.0f;
    for (int k = 0; k < K; ++k) {
        const uint32_t best = __reduce_max_sync(kAll, mine);
        if (best == 0u) break;
        const uint32_t e = __reduce_min_sync(kAll, mine == best ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
        const int owner = (int)(e & 31u);
        float l = 0.0f;
        if (lane == owner) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i == at) {
                    l = v[i];
                    key[i] = 0u;
                }
            local_best();
        }
        l = __shfl_sync(kAll, l, owner);
        if (lane == k) {
            my_id = (int)e;
            my_logit = l;
        }
    }
    float w = my_id >= 0 ? score(my_logit) : 0.0f;
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
