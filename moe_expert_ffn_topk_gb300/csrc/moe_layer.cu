// Host side of moe_layer (moe_ops.h): the workspace, the kernel's arguments and the choice of its format. The kernel is in
// moe_layer.cuh.
#include <algorithm>
#include <cmath>

#include "layer_parts.h"
#include "moe_layer.cuh"

namespace moe {

namespace layer {
extern template cudaError_t launch_fmt<MOE_LAYER_BF16>(const Args&, cudaStream_t);
extern template cudaError_t launch_fmt<MOE_LAYER_FP8_BLOCK>(const Args&, cudaStream_t);
extern template cudaError_t launch_fmt<MOE_LAYER_FP4_MX>(const Args&, cudaStream_t);
}  // namespace layer

namespace {

size_t align_up(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

LayerLayout layer_layout(const moe_dims& d, int weights) {
    const size_t T = d.num_tokens, R = T * (d.topk + d.num_shared_experts);
    LayerLayout L = {};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes);
        return at;
    };
    // the counters: the same place whatever the sizes, so that one workspace serves calls of different sizes
    L.header = take(sizeof(int32_t) * kOpsHeaderInts);
    L.dep = take(sizeof(int32_t) * layer::kMaxE);
    L.cols = take(sizeof(int32_t) * ((1 << 16) / 32));
    L.amax = take(sizeof(uint32_t) * layer::kMaxSlots);
    L.logits = take(sizeof(float) * T * d.num_experts);
    L.ids = take(sizeof(int32_t) * T * d.topk);
    L.weights = take(sizeof(float) * T * d.topk);
    L.x16 = take(2 * T * d.hidden);
    L.xinv = take(sizeof(float) * T);
    L.act = take(sizeof(float) * R * d.intermediate);
    L.comb = take(sizeof(float) * R * d.hidden * layer_parts(d, weights));
    L.total = off;
    return L;
}

cudaError_t launch_layer(const moe_layer_args& a, const moe_gate_options& gate, const moe_dims& d, void* workspace,
                         cudaStream_t s) {
    if (d.num_tokens == 0) return cudaSuccess;
    const LayerLayout L = layer_layout(d, a.weights);
    uint8_t* b = static_cast<uint8_t*>(workspace);
    layer::Args p = {};
    p.x = static_cast<const uint16_t*>(a.x);
    p.router = a.router;
    p.w1 = a.w1.data;
    p.w2 = a.w2.data;
    p.s1 = a.w1.scale;
    p.s2 = a.w2.scale;
    p.bias = a.gate_bias;
    p.ids_io = a.topk_ids;
    p.weights_io = a.topk_weights;
    p.y = static_cast<uint16_t*>(a.y);
    p.gate = gate;
    p.router_bf16 = a.router_type == MOE_TYPE_BF16;
    p.T = d.num_tokens;
    p.H = d.hidden;
    p.I = d.intermediate;
    p.E = d.num_experts;
    p.K = d.topk;
    p.S = d.num_shared_experts;
    p.clamp = a.has_activation_clamp ? a.activation_clamp : INFINITY;
    p.hdr = reinterpret_cast<int32_t*>(b + L.header);
    p.dep = reinterpret_cast<int32_t*>(b + L.dep);
    p.cols = reinterpret_cast<int32_t*>(b + L.cols);
    p.amax = reinterpret_cast<uint32_t*>(b + L.amax);
    p.logits = reinterpret_cast<float*>(b + L.logits);
    p.ids = reinterpret_cast<int32_t*>(b + L.ids);
    p.weights = reinterpret_cast<float*>(b + L.weights);
    p.x16 = reinterpret_cast<uint16_t*>(b + L.x16);
    p.xinv = reinterpret_cast<float*>(b + L.xinv);
    p.act = reinterpret_cast<float*>(b + L.act);
    p.comb = reinterpret_cast<float*>(b + L.comb);
    p.splits = layer_parts(d, a.weights);
    switch (a.weights) {
        case MOE_LAYER_BF16: return layer::launch_fmt<MOE_LAYER_BF16>(p, s);
        case MOE_LAYER_FP8_BLOCK: return layer::launch_fmt<MOE_LAYER_FP8_BLOCK>(p, s);
        default: return layer::launch_fmt<MOE_LAYER_FP4_MX>(p, s);
    }
}

}  // namespace moe
