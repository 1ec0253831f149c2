// Rows of x in int8 with a scale each (moe_int8_quantize in moe_ops.h). A CTA has a row: its values stay in registers between the largest
// magnitude and the codes, where they fit (rows of up to kThreads * 32 values), so x is read once. Bound by HBM: 2 (bf16) or 4 (fp32)
// bytes read and 1 written an element.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}

// kPer values of a thread from column c on (all of them, or the row's last ones)
template <typename T, int kPer>
__device__ __forceinline__ void load(const T* row, int64_t c, int64_t cols, float (&v)[kPer]) {
    if constexpr (kPer == 1) {
        v[0] = c < cols ? to_f32(row[c]) : 0.0f;
    } else {
        constexpr int kW = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < kPer / kW; ++j) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (c < cols) w = __ldg(reinterpret_cast<const uint4*>(row + c) + j);
            const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int k = 0; k < kW; ++k) v[j * kW + k] = to_f32(e[k]);
        }
    }
}

template <int kPer>
__device__ __forceinline__ void put(int8_t* row, int64_t c, int64_t cols, const float (&v)[kPer], float s) {
    if (c >= cols) return;
    uint32_t word[(kPer + 3) / 4] = {};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[j], s)), -127.0f), 127.0f);
        if (s < INFINITY) word[j / 4] |= ((uint32_t)(int)q & 0xffu) << (8 * (j % 4));
    }
    if constexpr (kPer == 1) row[c] = (int8_t)word[0];
    else *reinterpret_cast<uint2*>(row + c) = make_uint2(word[0], word[1]);
}

// kPer: values of a thread at a time (8 where rows of x start on 16 bytes, those of q on 8, and both have a multiple of 8 of
// them; else 1); kHold: how often it has some at most, 0: rows of any length, read twice
template <typename T, int kPer, int kHold>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t cols, int64_t x_stride, int8_t* __restrict__ q, int64_t q_stride,
                    float* __restrict__ scale, int64_t rows) {
    __shared__ uint32_t best[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* src = x + r * x_stride;
        // the largest magnitude as an integer: infinities and NaNs are above every number and survive
        uint32_t top = 0;
        auto look = [&](const float (&v)[kPer]) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        };
        float v[kHold > 0 ? kHold : 1][kPer];
        if constexpr (kHold > 0) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) load<T, kPer>(src, ((int64_t)h * kThreads + threadIdx.x) * kPer, cols, v[h]);
#pragma unroll
            for (int h = 0; h < kHold; ++h) look(v[h]);
        } else {
            for (int64_t c = threadIdx.x * kPer; c < cols; c += kThreads * kPer) {
                load<T, kPer>(src, c, cols, v[0]);
                look(v[0]);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) best[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) top = max(top, best[w]);
        __syncthreads();
        float s = __fdiv_rn(__uint_as_float(top), 127.0f);
        if (s < 1e-8f) s = 1e-8f;
        if (threadIdx.x == 0) scale[r] = s;
        if constexpr (kHold > 0) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) put<kPer>(q + r * q_stride, ((int64_t)h * kThreads + threadIdx.x) * kPer, cols, v[h], s);
        } else {
            for (int64_t c = threadIdx.x * kPer; c < cols; c += kThreads * kPer) {
                load<T, kPer>(src, c, cols, v[0]);
                put<kPer>(q + r * q_stride, c, cols, v[0], s);
            }
        }
    }
}

template <typename T>
cudaError_t launch(const T* x, int64_t rows, int64_t cols, int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                   cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(rows, 0x7fffffff);
    const bool vec = !((reinterpret_cast<uintptr_t>(x) | (uint64_t)(x_stride * (int64_t)sizeof(T))) & 15) &&
                     !((reinterpret_cast<uintptr_t>(q) | (uint64_t)q_stride | (uint64_t)cols) & 7);
#define MOE_QUANT(per, hold) quantize_kernel<T, per, hold><<<grid, kThreads, 0, s>>>(x, cols, x_stride, q, q_stride, scale, rows)
    const int64_t times = (cols + kThreads * (vec ? 8 : 1) - 1) / (kThreads * (vec ? 8 : 1));
    if (vec) {
        if (times <= 1) MOE_QUANT(8, 1);
        else if (times <= 2) MOE_QUANT(8, 2);
        else if (times <= 4) MOE_QUANT(8, 4);
        else MOE_QUANT(8, 0);
    } else {
        if (times <= 8) MOE_QUANT(1, 8);
        else if (times <= 32) MOE_QUANT(1, 32);
        else MOE_QUANT(1, 0);
    }
#undef MOE_QUANT
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, int8_t* q,
                                 int64_t q_stride, float* scale, cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    if (type == MOE_TYPE_BF16) return launch(static_cast<const __nv_bfloat16*>(x), rows, cols, x_stride, q, q_stride, scale, s);
    return launch(static_cast<const float*>(x), rows, cols, x_stride, q, q_stride, scale, s);
}

}  // namespace moe
