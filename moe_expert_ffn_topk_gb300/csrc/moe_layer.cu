// The whole MoE layer for a few tokens (moe_layer in moe_ops.h).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"

namespace moe {

namespace {

struct Args {
    moe_layer_args a;
    int T, H, I, E, K, S;
    float clamp;
    int32_t* hdr;
    float *logits, *weights, *act, *slots;
    int32_t* ids;
};

// Weight (n, k) of expert e, layer 1 or 2, as fp32.
template <int kFmt>
__device__ __forceinline__ float weight(const moe_operand& w, int e, int n, int k, int N, int Kd) {
    if constexpr (kFmt == MOE_LAYER_BF16) {
        return bf16_bits_to_float(static_cast<const uint16_t*>(w.data)[((int64_t)e * Kd + k) * N + n]);
    } else if constexpr (kFmt == MOE_LAYER_FP8_BLOCK) {
        const float s = static_cast<const float*>(w.scale)[((int64_t)e * (N / 128) + n / 128) * (Kd / 128) + k / 128];
        return e4m3_to_float(static_cast<const uint8_t*>(w.data)[((int64_t)e * N + n) * Kd + k]) * s;
    } else {
        const int64_t row = (int64_t)e * N + n;
        const uint8_t b = static_cast<const uint8_t*>(w.data)[row * (Kd / 2) + k / 2];
        return e2m1_to_float(k & 1 ? b >> 4 : b & 15) * ue8m0_to_float(static_cast<const uint8_t*>(w.scale)[row * (Kd / 32) + k / 32]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__global__ void logits_kernel(Args p) {
    const int w = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x & 31;
    if (w >= p.T * p.E) return;
    const int t = w / p.E, e = w % p.E;
    float sum = 0.0f;
    for (int h = lane; h < p.H; h += 32) {
        const float r = p.a.router_type == MOE_TYPE_BF16
                            ? bf16_bits_to_float(static_cast<const uint16_t*>(p.a.router)[(int64_t)e * p.H + h])
                            : static_cast<const float*>(p.a.router)[(int64_t)e * p.H + h];
        sum = fmaf(bf16_bits_to_float(static_cast<const uint16_t*>(p.a.x)[(int64_t)t * p.H + h]), r, sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) p.logits[(int64_t)t * p.E + e] = sum;
}

__device__ __forceinline__ int slot_expert(const Args& p, int t, int k) {
    if (k >= p.K) return p.E + k - p.K;
    const int e = p.ids[t * p.K + k];
    if (e < -1 || e >= p.E) {
        record_error(p.hdr, MOE_ERR_BAD_ROUTE);
        return -1;
    }
    return e;
}

template <int kFmt>
__global__ void up_kernel(Args p) {
    const int w = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x & 31;
    const int Kt = p.K + p.S;
    if (w >= p.T * Kt * p.I) return;
    const int slot = w / p.I, j = w % p.I, t = slot / Kt;
    const int e = slot_expert(p, t, slot % Kt);
    if (e < 0) return;
    float g = 0.0f, u = 0.0f;
    for (int h = lane; h < p.H; h += 32) {
        const float x = bf16_bits_to_float(static_cast<const uint16_t*>(p.a.x)[(int64_t)t * p.H + h]);
        g = fmaf(x, weight<kFmt>(p.a.w1, e, j, h, 2 * p.I, p.H), g);
        u = fmaf(x, weight<kFmt>(p.a.w1, e, p.I + j, h, 2 * p.I, p.H), u);
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) p.act[(int64_t)slot * p.I + j] = swiglu1(g, u, p.clamp);
}

template <int kFmt>
__global__ void down_kernel(Args p) {
    const int w = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x & 31;
    const int Kt = p.K + p.S;
    if (w >= p.T * p.H) return;
    const int t = w / p.H, h = w % p.H;
    float y = 0.0f;
    for (int k = 0; k < Kt; ++k) {
        const int e = slot_expert(p, t, k);
        if (e < 0) continue;
        float sum = 0.0f;
        for (int i = lane; i < p.I; i += 32)
            sum = fmaf(p.act[(int64_t)(t * Kt + k) * p.I + i], weight<kFmt>(p.a.w2, e, h, i, p.H, p.I), sum);
        sum = warp_sum(sum);
        y += k < p.K ? p.weights[t * p.K + k] * sum : sum;
    }
    if (lane == 0) static_cast<uint16_t*>(p.a.y)[(int64_t)t * p.H + h] = float_to_bf16_bits(y);
}

template <int kFmt>
cudaError_t launch_ffn(const Args& p, cudaStream_t s) {
    up_kernel<kFmt><<<(unsigned)(((int64_t)p.T * (p.K + p.S) * p.I + 7) / 8), 256, 0, s>>>(p);
    down_kernel<kFmt><<<(unsigned)(((int64_t)p.T * p.H + 7) / 8), 256, 0, s>>>(p);
    return cudaGetLastError();
}

size_t align_up(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

LayerLayout layer_layout(const moe_dims& d) {
    const size_t T = d.num_tokens, R = T * (d.topk + d.num_shared_experts);
    LayerLayout L = {};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes);
        return at;
    };
    L.header = take(sizeof(int32_t) * kOpsHeaderInts);
    L.logits = take(sizeof(float) * T * d.num_experts);
    L.ids = take(sizeof(int32_t) * T * d.topk);
    L.weights = take(sizeof(float) * T * d.topk);
    L.act = take(sizeof(float) * R * d.intermediate);
    L.total = off;
    return L;
}

cudaError_t launch_layer(const moe_layer_args& a, const moe_gate_options& gate, const moe_dims& d, void* workspace,
                         cudaStream_t s) {
    if (d.num_tokens == 0) return cudaSuccess;
    const LayerLayout L = layer_layout(d);
    uint8_t* b = static_cast<uint8_t*>(workspace);
    Args p = {};
    p.a = a;
    p.T = d.num_tokens;
    p.H = d.hidden;
    p.I = d.intermediate;
    p.E = d.num_experts;
    p.K = d.topk;
    p.S = d.num_shared_experts;
    p.clamp = a.has_activation_clamp ? a.activation_clamp : INFINITY;
    p.hdr = reinterpret_cast<int32_t*>(b + L.header);
    p.logits = reinterpret_cast<float*>(b + L.logits);
    p.act = reinterpret_cast<float*>(b + L.act);
    p.ids = a.topk_ids ? a.topk_ids : reinterpret_cast<int32_t*>(b + L.ids);
    p.weights = a.topk_weights ? a.topk_weights : reinterpret_cast<float*>(b + L.weights);
    if (a.router) {
        logits_kernel<<<(p.T * p.E + 7) / 8, 256, 0, s>>>(p);
        const cudaError_t e = launch_gate(p.logits, MOE_TYPE_F32, p.E, a.gate_bias, gate, p.T, p.E, p.K, p.ids, p.weights, s);
        if (e != cudaSuccess) return e;
    }
    switch (a.weights) {
        case MOE_LAYER_BF16: return launch_ffn<MOE_LAYER_BF16>(p, s);
        case MOE_LAYER_FP8_BLOCK: return launch_ffn<MOE_LAYER_FP8_BLOCK>(p, s);
        default: return launch_ffn<MOE_LAYER_FP4_MX>(p, s);
    }
}

}  // namespace moe
