// Rows of x in e4m3 with an fp32 scale for each 128 columns (moe_fp8_quantize in moe_ops.h).
//
// One pass: 8 lanes hold a block of 128 columns, 16 values each, so the block's amax is three shuffles and x is read
// once. Bound by HBM: 2 (bf16) or 4 (fp32) bytes read and 1 written an element. That takes the division out of the way: by a
// power of two it is an exact product, and by other scales it is Markstein's: with r = 1/s rounded to nearest, q = x r and
// q - r (q s - x) with fused multiply-adds is x / s rounded to nearest, wherever nothing over- or underflows (scales outside
// 2^-60 .. 2^60 take the division itself). 8192 x 7168 bf16 to power-of-two scales: 31.7 us, 0.84 of the
// copy rate (51 us with a division a value, 41 before the resident grid with the next unit's loads in flight); to other scales 37.2,
// 0.72. From fp32 59.3 and 61.0 us, 0.75 and 0.73.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

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

// two e4m3 codes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(hi), "f"(lo));
    return pair;
}

// kVec: rows of x are 16-byte aligned and of q too, so every full lane loads and stores 16 bytes at a time. Index: of a unit of
// four blocks (a warp's), 32 bits wide where they suffice.
template <typename T, bool kPow2, bool kVec, typename Index>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t cols, int64_t x_stride, uint8_t* __restrict__ q, int64_t q_stride,
                    float* __restrict__ scale, Index blocks, Index units_per_row, Index units) {
    const int sub = threadIdx.x % kLanes;
    const Index first = (Index)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, step = (Index)gridDim.x * (kThreads / 32);
    constexpr int kW = 16 / sizeof(T);
    // where unit u's lane begins, and how many values it has there
    Index r, b;
    int64_t c0;
    int n;
    auto place = [&](Index u) {
        r = u / units_per_row;
        b = (u - r * units_per_row) * 4 + (threadIdx.x & 31) / kLanes;
        c0 = (int64_t)b * 128 + sub * kPer;
        n = u < units ? (int)max((int64_t)0, min((int64_t)kPer, cols - c0)) : 0;
    };
    uint4 w[kPer / kW];  // of a full lane: the next unit's values are on their way while one is worked on
    auto load = [&]() {
        const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)r * x_stride + c0);
#pragma unroll
        for (int j = 0; j < kPer / kW; ++j) w[j] = __ldg(src + j);
    };
    place(first);
    if (kVec && n == kPer) load();
    for (Index u = first; u < units; u += step) {
        place(u);
        const Index row = r, block = b;
        const int64_t col = c0;
        const int have = n;
        float v[kPer];
        if (kVec && have == kPer) {
#pragma unroll
            for (int j = 0; j < kPer / kW; ++j) {
                const T* e = reinterpret_cast<const T*>(&w[j]);
#pragma unroll
                for (int k = 0; k < kW; ++k) v[j * kW + k] = to_f32(e[k]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = j < have ? to_f32(x[(int64_t)row * x_stride + col + j]) : 0.0f;
        }
        place(u + step);
        if (kVec && n == kPer) load();
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
        if (have == 0) continue;
        if (sub == 0) scale[(int64_t)row * blocks + block] = s;
        uint32_t word[kPer / 4];
        auto code = [&](auto quotient) {
#pragma unroll
            for (int j = 0; j < kPer; j += 4)
                word[j / 4] = e4m3x2(quotient(v[j]), quotient(v[j + 1])) | (e4m3x2(quotient(v[j + 2]), quotient(v[j + 3])) << 16);
        };
        if (s > 8.6736174e-19f && s < 1.1529215e18f) {  // 2^-60, 2^60
            // (of a power of two: the exponent turned round)
            const float inv = kPow2 ? __uint_as_float(0x7f000000u - __float_as_uint(s)) : __fdiv_rn(1.0f, s);
            if constexpr (kPow2) {
                code([&](float x) { return __fmul_rn(x, inv); });
            } else {
                // the residual with the other sign: that of a zero x is +0, and -inv times it -0, which leaves y's own sign (with
                // x - y s and inv, -0 came out as +0)
                code([&](float x) {
                    const float y = __fmul_rn(x, inv);
                    return __fmaf_rn(__fmaf_rn(y, s, -x), -inv, y);
                });
            }
        } else {
            code([&](float x) { return __fdiv_rn(x, s); });
        }
        uint8_t* dst = q + (int64_t)row * q_stride + col;
        if (kVec && have == kPer) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (j < have) dst[j] = (uint8_t)(word[j / 4] >> (8 * (j % 4)));
        }
    }
}

template <typename T, bool kPow2>
cudaError_t launch(const void* x, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* q, int64_t q_stride, float* scale,
                   cudaStream_t s) {
    const int64_t blocks = (cols + 127) / 128, per_row = (blocks + 3) / 4, units = rows * per_row;
    const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
    // what the SMs hold at a time of the bf16 kernel on 32-bit numbers (48 registers); of the fp32 ones (61-64) they hold four, and a
    // fifth of the shares runs after the others
    const int grid = (int)std::min<int64_t>(ctas, (int64_t)tc_num_sms() * 5);
    const bool vec = !((reinterpret_cast<uintptr_t>(x) | (uint64_t)(x_stride * (int64_t)sizeof(T)) |
                        reinterpret_cast<uintptr_t>(q) | (uint64_t)q_stride) & 15);
    const T* xt = static_cast<const T*>(x);
    // 32-bit unit numbers, the step past the last one included; sizes beyond them are odd enough for the slower rows
    if (units < (int64_t(1) << 31) && vec)
        quantize_kernel<T, kPow2, true, uint32_t><<<grid, kThreads, 0, s>>>(xt, cols, x_stride, q, q_stride, scale, (uint32_t)blocks,
                                                                            (uint32_t)per_row, (uint32_t)units);
    else if (vec)
        quantize_kernel<T, kPow2, true, uint64_t><<<grid, kThreads, 0, s>>>(xt, cols, x_stride, q, q_stride, scale, (uint64_t)blocks,
                                                                            (uint64_t)per_row, (uint64_t)units);
    else
        quantize_kernel<T, kPow2, false, uint64_t><<<grid, kThreads, 0, s>>>(xt, cols, x_stride, q, q_stride, scale, (uint64_t)blocks,
                                                                             (uint64_t)per_row, (uint64_t)units);
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
