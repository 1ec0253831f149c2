// The router (moe_gate in moe_ops.h): expert ids and gate weights from logits, one warp per token.
//
// A row of up to 1024 logits is read once, into shared memory, and every step after that is a reduction over the warp: the
// maximum and sum of the softmax, the two best of every group, and K rounds of "largest key, lowest index" (two warp-wide
// integer reductions each). Bound by those chains' latency, not by HBM: 7 tokens x 256 experts (sigmoid, bias, groups, top-8) 5.1 us on
// the device (a warp by itself, instructions cached: 1000 cycles to read the row, 1300 for the scores, 1500 for the groups, 3000 for
// the rounds, 1100 for the weights); 8192 x 60 (softmax, top-4) 10.2 us.
#include "gate_select.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;  // tokens per CTA, while their rows fit 48 KB

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
    if constexpr (sizeof(T) == 2) return bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(p));
    else return *p;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    gate_kernel(const T* __restrict__ logits, int64_t stride, const float* __restrict__ bias, moe_gate_options o, int tokens,
                int E, int K, int32_t* __restrict__ ids, float* __restrict__ weights) {
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= tokens) return;
    const T* row = logits + (int64_t)t * stride;
    float* scratch = smem + warp * gate_scratch(E);
#pragma unroll 8
    for (int e = lane; e < E; e += 32) scratch[e] = load_logit(row + e);
    if (bias)
#pragma unroll 8
        for (int e = lane; e < E; e += 32) scratch[E + e] = __ldg(bias + e);
    gate_token(scratch, bias != nullptr, o, E, K, lane, ids + (int64_t)t * K, weights + (int64_t)t * K);
}

template <typename T>
cudaError_t launch_t(const void* logits, int64_t stride, const float* bias, const moe_gate_options& o, int T_, int E, int K,
                     int32_t* ids, float* weights, cudaStream_t s) {
    const int warps = E <= 512 ? kWarps : kWarps / 2;
    const size_t smem = sizeof(float) * warps * gate_scratch(E);
    gate_kernel<T><<<(T_ + warps - 1) / warps, 32 * warps, smem, s>>>(static_cast<const T*>(logits), stride, bias, o, T_, E, K, ids,
                                                                        weights);
    return cudaGetLastError();
}

}  // namespace

bool gate_options_ok(const moe_gate_options& o, int E, int K) {
    if (o.score != MOE_SCORE_SOFTMAX && o.score != MOE_SCORE_SIGMOID) return false;
    if (o.num_groups < 1 || o.num_groups > 32 || E % o.num_groups) return false;
    if (o.topk_groups < 1 || o.topk_groups > o.num_groups || (int64_t)o.topk_groups * (E / o.num_groups) < K) return false;
    if (o.group_top != 1 && o.group_top != 2) return false;
    return o.route_scale - o.route_scale == 0.0f;  // finite
}

cudaError_t launch_gate(const void* logits, int type, int64_t stride, const float* bias, const moe_gate_options& o, int T,
                        int E, int K, int32_t* ids, float* weights, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    if (type == MOE_TYPE_BF16) return launch_t<__nv_bfloat16>(logits, stride, bias, o, T, E, K, ids, weights, s);
    return launch_t<float>(logits, stride, bias, o, T, E, K, ids, weights, s);
}

}  // namespace moe
