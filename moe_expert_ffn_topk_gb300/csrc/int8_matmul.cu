// Product of int8 matrices with a scale for each row of either (moe_int8_matmul in moe_ops.h).
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

template <typename Out>
__global__ void __launch_bounds__(256) simple_kernel(moe_int8_matmul_args p) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        int g = 0;
        if (p.offsets) {
            int end = min(max(__ldg(p.offsets), 0), (int)p.M);
            for (g = 0; g < p.groups; ++g) {
                end = max(end, min(max(__ldg(p.offsets + g + 1), 0), (int)p.M));
                if (m < end) break;
            }
            if (g == p.groups || m < min(max(__ldg(p.offsets), 0), (int)p.M)) continue;
        }
        const uint4* a = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.a) + m * p.a_stride);
        const uint4* b = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.b) + (g * p.N + n) * p.b_stride);
        int c = 0;
        for (int64_t k = 0; k < p.K / 16; ++k) {
            const uint4 u = __ldg(a + k), v = __ldg(b + k);
            c = __dp4a((int)u.x, (int)v.x, c);
            c = __dp4a((int)u.y, (int)v.y, c);
            c = __dp4a((int)u.z, (int)v.z, c);
            c = __dp4a((int)u.w, (int)v.w, c);
        }
        const float y = __fmul_rn(__fmul_rn((float)c, __ldg(p.b_scale + (int64_t)g * p.N + n)), __ldg(p.a_scale + m));
        if constexpr (sizeof(Out) == 2) static_cast<uint16_t*>(p.out)[m * p.out_stride + n] = float_to_bf16_bits(y);
        else static_cast<float*>(p.out)[m * p.out_stride + n] = y;
    }
}

}  // namespace

size_t int8_matmul_workspace(int64_t, int64_t, int64_t, int) { return sizeof(int32_t) * kOpsHeaderInts; }

cudaError_t launch_int8_matmul(const moe_int8_matmul_args& a, void*, cudaStream_t s) {
    const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)std::min<int64_t>(a.M, 65535));
    if (a.out_type == MOE_TYPE_BF16) simple_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else simple_kernel<float><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
