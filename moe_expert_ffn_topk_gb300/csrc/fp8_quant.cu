// Rows of x in e4m3 with an fp32 scale for each 128 columns (moe_fp8_quantize in moe_ops.h).
//
// One pass: 8 lanes hold a block of 128 columns, 16 values each, so the block's amax is three shuffles and x is read
// once. Bound by HBM: 2 (bf16) or 4 (fp32) bytes read and 1 written an element.
#include "common.cuh"
#include "ops.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                 // values of a lane
constexpr int kLanes = 128 / kPer;       // lanes of a block of 128 columns

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}

// kVec: rows of x are 16-byte aligned and of q too, so every full lane loads and stores 16 bytes at a time
template <typename T, bool kPow2, bool kVec>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* __restrict__ q,
                    int64_t q_stride, float* __restrict__ scale, int64_t blocks) {
    const int64_t total = rows * blocks;
    const int sub = threadIdx.x % kLanes;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;; i += (int64_t)gridDim.x * kThreads / kLanes) {
        const bool on = i < total;
        if (!__any_sync(0xffffffffu, on)) break;  // whole warps leave together
        const int64_t r = on ? i / blocks : 0, b = on ? i % blocks : 0;
        const int64_t c0 = b * 128 + sub * kPer;
        const int n = on ? (int)max((int64_t)0, min((int64_t)kPer, cols - c0)) : 0;
        const T* src = x + r * x_stride + c0;
        float v[kPer];
        if (kVec && n == kPer) {
            constexpr int kW = 16 / sizeof(T);
#pragma unroll
            for (int j = 0; j < kPer / kW; ++j) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + j);
                const T* p = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int k = 0; k < kW; ++k) v[j * kW + k] = to_f32(p[k]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = j < n ? to_f32(src[j]) : 0.0f;
        }
        // the largest magnitude as an integer: infinities and NaNs are above every number and survive
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
        for (int d = kLanes / 2; d >= 1; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        float s = __fdiv_rn(__uint_as_float(top), 448.0f);
        // the next power of two: any fraction bit carries into the exponent (not of an infinity or NaN)
        if (kPow2 && top < 0x7f800000u) s = __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
        if (s == 0.0f) s = 1.0f;
        if (!on) continue;
        if (sub == 0) scale[r * blocks + b] = s;
        uint8_t* dst = q + r * q_stride + c0;
        uint32_t word[kPer / 4];
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w |= (uint32_t)float_to_e4m3_satfinite(__fdiv_rn(v[j + k], s)) << (8 * k);
            word[j / 4] = w;
        }
        if (kVec && n == kPer) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (j < n) dst[j] = (uint8_t)(word[j / 4] >> (8 * (j % 4)));
        }
    }
}

template <typename T, bool kPow2>
cudaError_t launch(const void* x, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* q, int64_t q_stride, float* scale,
                   cudaStream_t s) {
    const int64_t blocks = (cols + 127) / 128;
    const int64_t ctas = (rows * blocks * kLanes + kThreads - 1) / kThreads;
    const int grid = (int)(ctas < (1 << 20) ? ctas : (1 << 20));
    const bool vec = !((reinterpret_cast<uintptr_t>(x) | (uint64_t)(x_stride * (int64_t)sizeof(T)) |
                        reinterpret_cast<uintptr_t>(q) | (uint64_t)q_stride) & 15);
    const T* xt = static_cast<const T*>(x);
    if (vec) quantize_kernel<T, kPow2, true><<<grid, kThreads, 0, s>>>(xt, rows, cols, x_stride, q, q_stride, scale, blocks);
    else quantize_kernel<T, kPow2, false><<<grid, kThreads, 0, s>>>(xt, rows, cols, x_stride, q, q_stride, scale, blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* q,
                                int64_t q_stride, float* scale, bool pow2, cudaStream_t s) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    if (type == MOE_TYPE_BF16)
        return pow2 ? launch<__nv_bfloat16, true>(x, rows, cols, x_stride, q, q_stride, scale, s)
                    : launch<__nv_bfloat16, false>(x, rows, cols, x_stride, q, q_stride, scale, s);
    return pow2 ? launch<float, true>(x, rows, cols, x_stride, q, q_stride, scale, s)
                : launch<float, false>(x, rows, cols, x_stride, q, q_stride, scale, s);
}

}  // namespace moe
