// Declarations shared by the operators of moe_ops.h: the launchers and the layout of their workspaces.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "moe_ops.h"

namespace moe {

// The head of an operator's workspace: [0] is the error word that moe_check_device_error reads; the rest are
// counters that every call leaves at zero.
constexpr int kOpsHeaderInts = 64;

// Experts of a router and selected experts per token that fit a warp's registers.
constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxTopk = 32;

inline moe_gate_options default_gate_options() {
    moe_gate_options o = {};
    o.score = MOE_SCORE_SOFTMAX;
    o.num_groups = o.topk_groups = o.group_top = o.normalize = 1;
    o.route_scale = 1.0f;
    return o;
}
// setmaxnreg hands out the registers that a launch holds; a split made for `regs` a thread would wait for ever in a build of the
// kernel that holds fewer, so such a build is refused before its first launch.
inline cudaError_t check_register_split(const void* kernel, int regs) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    return e != cudaSuccess ? e : a.numRegs >= regs ? cudaSuccess : cudaErrorLaunchOutOfResources;
}

// What has to be done once before a kernel's first launch on a device (its attributes belong to the device that is current when they are
// set): calls set(device) the first time on each and returns what it returned there. *device: the current one. Set is a lambda of the
// one place that uses it.
constexpr int kMaxDevices = 64;
template <typename Set>
cudaError_t once_per_device(int* device, Set set) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    const cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess) return e;
    const int d = *device;
    if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[d], [&] { err[d] = set(d); });
    return err[d];
}

bool gate_options_ok(const moe_gate_options& o, int E, int K);

cudaError_t launch_gate(const void* logits, int type, int64_t stride, const float* bias, const moe_gate_options& o, int T,
                        int E, int K, int32_t* ids, float* weights, cudaStream_t s);
cudaError_t launch_fp8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* q,
                                int64_t q_stride, float* scale, bool pow2, cudaStream_t s);
size_t fp8_matmul_workspace(int64_t M, int64_t N, int64_t K, int groups);
cudaError_t launch_fp8_matmul(const moe_fp8_matmul_args& a, void* workspace, cudaStream_t s);

// Slots (tokens x K) of a routing call, its experts and the experts of one token.
constexpr int64_t kMaxSlots = int64_t(1) << 24;
constexpr int kRowExperts = 1024, kRowTopk = 32;
size_t permute_workspace(int64_t T, int K, int E);
cudaError_t launch_permute(const moe_permute_args& a, int T, int K, int E, int32_t* hdr, cudaStream_t s);

struct UnpermuteArgs {
    const void* rows;  // [T*K, H]
    const int32_t* slot_row;
    const float* weights;
    const void* dy;    // backward
    void* out;         // y, or d_rows
    float* d_weights;
    int64_t H, rows_stride, dy_stride, out_stride;
    int T, K, type, token_type;  // of the rows (and d_rows); of y and dy
};
cudaError_t launch_unpermute(const UnpermuteArgs& a, cudaStream_t s);
cudaError_t launch_unpermute_backward(const UnpermuteArgs& a, cudaStream_t s);

cudaError_t launch_int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, int8_t* q,
                                 int64_t q_stride, float* scale, cudaStream_t s);
size_t int8_matmul_workspace(int64_t M, int64_t N, int64_t K, int groups);
cudaError_t launch_int8_matmul(const moe_int8_matmul_args& a, void* workspace, cudaStream_t s);

// Byte offsets of moe_layer's workspace.
struct LayerLayout {
    size_t header, dep, cols, amax, logits, ids, weights, x16, xinv, act, comb, total;
};
LayerLayout layer_layout(const moe_dims& d, int weights);
cudaError_t launch_layer(const moe_layer_args& a, const moe_gate_options& gate, const moe_dims& d, void* workspace,
                         cudaStream_t s);

}  // namespace moe
