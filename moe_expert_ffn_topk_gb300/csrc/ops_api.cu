// Host side of the operators of moe_ops.h: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "ops.h"

using namespace moe;

namespace {

moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool type_ok(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

int type_bytes(int32_t t) { return t == MOE_TYPE_BF16 ? 2 : 4; }

bool workspace_ok(const void* ws, size_t have, size_t need) { return ws && aligned(ws, 256) && have >= need; }

// x 2^62: products of the sizes stay inside 64 bits
bool extent_ok(int64_t rows, int64_t stride) { return stride >= 0 && (rows == 0 || stride <= (int64_t(1) << 62) / rows); }

// M: a tile of 256 rows may begin at any row, and its last row's number stays inside 32 bits
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;

bool matmul_sizes_ok(int64_t M, int64_t N, int64_t K, int32_t groups) {
    return M >= 0 && M <= kMaxRows && N >= 1 && N <= (1 << 20) && K >= 16 && K <= (1 << 20) && K % 16 == 0 &&
           groups >= 1 && groups <= 1024;
}

bool layer_dims_ok(const moe_dims* d, int weights) {
    return dims_ok(d, MOE_A16W16) && weights >= MOE_LAYER_BF16 && weights <= MOE_LAYER_FP4_MX;
}

}  // namespace

extern "C" {

moe_status moe_ops_workspace_init(void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!workspace || !aligned(workspace, 256)) return MOE_ERR_WORKSPACE;
    return from_cuda(cudaMemsetAsync(workspace, 0, workspace_bytes, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_gate(const void* logits, moe_type type, int64_t row_stride, const float* bias, const moe_gate_options* opt,
                    const moe_dims* d, int32_t* topk_ids, float* topk_weights, moe_stream_t stream) {
    if (!d || !type_ok(type) || d->num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const int T = d->num_tokens, E = d->num_experts, K = d->topk;
    if (K < 1 || K > kGateMaxTopk || E < K || E > kGateMaxExperts || (int64_t)T * K > (int64_t(1) << 24))
        return MOE_ERR_INVALID_ARG;
    const moe_gate_options o = opt ? *opt : default_gate_options();
    if (!gate_options_ok(o, E, K) || row_stride < E || !extent_ok(T, row_stride)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_weights || !aligned(logits, type_bytes(type)) || !aligned(bias, 4) ||
        !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_gate(logits, type, row_stride, bias, o, T, E, K, topk_ids, topk_weights,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_quantize(const void* x, moe_type type, int64_t rows, int64_t cols, int64_t x_stride, void* q,
                            int64_t q_stride, float* scale, uint32_t flags, moe_stream_t stream) {
    if (!type_ok(type) || rows < 0 || cols < 0 || (cols == 0 && rows > 0) || x_stride < cols || q_stride < cols ||
        (flags & ~(uint32_t)MOE_QUANT_POW2) || cols >= (int64_t(1) << 40) || !extent_ok(rows, x_stride) ||
        !extent_ok(rows, q_stride))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !scale || !aligned(x, type_bytes(type)) || !aligned(scale, 4)) return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_fp8_quantize(x, type, rows, cols, x_stride, static_cast<uint8_t*>(q), q_stride, scale,
                                         flags & MOE_QUANT_POW2, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t groups) {
    return matmul_sizes_ok(M, N, K, groups) ? fp8_matmul_workspace(M, N, K, groups) : 0;
}

moe_status moe_fp8_matmul(const moe_fp8_matmul_args* a, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!a || !matmul_sizes_ok(a->M, a->N, a->K, a->groups) || !type_ok(a->out_type)) return MOE_ERR_INVALID_ARG;
    if (a->a_stride < a->K || a->b_stride < a->K || a->out_stride < a->N || a->a_stride % 16 || a->b_stride % 16)
        return MOE_ERR_INVALID_ARG;
    if (!extent_ok(a->M, a->a_stride) || !extent_ok(a->N * a->groups, a->b_stride) || !extent_ok(a->M, a->out_stride))
        return MOE_ERR_INVALID_ARG;
    if (a->groups > 1 && !a->offsets) return MOE_ERR_INVALID_ARG;
    if (a->M == 0) return MOE_OK;
    if (!a->a || !a->a_scale || !a->b || !a->b_scale || !a->out || !aligned(a->a, 16) || !aligned(a->b, 16) ||
        !aligned(a->a_scale, 4) || !aligned(a->b_scale, 4) || !aligned(a->offsets, 4) || !aligned(a->out, type_bytes(a->out_type)))
        return MOE_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, fp8_matmul_workspace(a->M, a->N, a->K, a->groups))) return MOE_ERR_WORKSPACE;
    return from_cuda(launch_fp8_matmul(*a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_layer_workspace_bytes(const moe_dims* d, moe_layer_weights weights) {
    if (!layer_dims_ok(d, weights) || d->num_tokens > MOE_LAYER_MAX_TOKENS) return 0;
    // K is cut into more parts for fewer tokens, which can take more memory: enough for any number up to this one
    size_t most = 0;
    for (moe_dims few = *d; few.num_tokens >= 0; --few.num_tokens) most = std::max(most, layer_layout(few, weights).total);
    return most;
}

moe_status moe_layer(const moe_layer_args* a, const moe_dims* d, void* workspace, size_t workspace_bytes,
                     moe_stream_t stream) {
    if (!a || !layer_dims_ok(d, a->weights)) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > MOE_LAYER_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (a->has_activation_clamp && !(a->activation_clamp >= 0.0f)) return MOE_ERR_INVALID_ARG;
    const moe_gate_options o = a->gate ? *a->gate : default_gate_options();
    if (a->router && (!type_ok(a->router_type) || !gate_options_ok(o, d->num_experts, d->topk))) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens == 0) return MOE_OK;
    if (!a->x || !a->y || !a->w1.data || !a->w2.data) return MOE_ERR_INVALID_ARG;
    if (a->weights != MOE_LAYER_BF16 && (!a->w1.scale || !a->w2.scale)) return MOE_ERR_INVALID_ARG;
    if (!a->router && (!a->topk_ids || !a->topk_weights)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {a->x, a->router, a->w1.data, a->w1.scale, a->w2.data, a->w2.scale, (const void*)a->y})
        if (!aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a->topk_ids, 4) || !aligned(a->topk_weights, 4) || !aligned(a->gate_bias, 4)) return MOE_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, layer_layout(*d, a->weights).total)) return MOE_ERR_WORKSPACE;
    return from_cuda(launch_layer(*a, o, *d, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
