// How moe_layer cuts K of its second product into parts: arithmetic on the sizes alone (no CUDA headers), shared by the
// workspace's size, the launch, the kernel and the tests.
#pragma once

#include <algorithm>
#include <cstdint>

#include "moe_ops.h"

namespace moe {

// Stages of a part where `steps` stages are cut into `parts` (the last one may have fewer).
constexpr int part_steps(int steps, int parts) { return (steps + parts - 1) / parts; }

// SMs of the GPU the rule is made for. A constant, as the workspace's size follows from it and may be asked for without a GPU.
constexpr int kPartSms = 152;

// As many parts as give every SM a dozen units where few experts have rows (they are handed out one by one, so a unit is what the
// SMs can be apart at the end), of at least four stages each but for the last. Every part has a stage: the kernel's queue of units
// counts on it (kLead in moe_layer.cuh).
inline int layer_parts(const moe_dims& d, int weights) {
    const int64_t columns = d.hidden / (weights == MOE_LAYER_BF16 ? 128 : 32);
    const int64_t experts = std::min<int64_t>(d.num_experts, (int64_t)d.num_tokens * d.topk) + d.num_shared_experts;
    const int64_t step = weights == MOE_LAYER_BF16 ? 64 : weights == MOE_LAYER_FP8_BLOCK ? 256 : 512;
    const int steps = (int)((d.intermediate + step - 1) / step);
    if (columns * experts == 0) return 1;
    const int64_t want = (12 * kPartSms + columns * experts - 1) / (columns * experts);
    const int64_t most = std::max<int64_t>(1, d.intermediate / step / 4);
    const int parts = (int)std::min<int64_t>(std::min(want, most), 16), each = part_steps(steps, parts);
    // whole stages a part can leave the last parts with none (40 stages in 9 parts are 8 of 5): those are dropped
    return (steps + each - 1) / each;
}

}  // namespace moe
