// Rows of x in int8 with a scale each (moe_int8_quantize in moe_ops.h). A CTA has a row, or lanes of a warp where rows are short and many:
// its values stay in registers between the largest magnitude and the codes, where they fit, so x is read once. Bound by HBM: 2 (bf16)
// or 4 (fp32) bytes read and 1 written an element. That takes the division out of the way: x / s is Markstein's quotient from r = 1/s rounded to nearest (y = x r, then
// y + r (x - y s) with fused multiply-adds is x / s rounded to nearest wherever nothing under- or overflows; s >= 1e-8 and
// r >= 2^-122, so that only quotients far below one half do, whose code is 0 all the same), and adding 1.5 * 2^23 rounds it half to
// even into the low bits. |x| / s is at most 127 (1 + 2^-22), so no code passes 127.
// 8192 x 7168 bf16: 28.4 us, 0.93 of the copy rate (66 us with a division a value).
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

// kPer values of a thread, as they lie in memory: kVec 16 bytes of x, else one value
template <typename T, bool kVec>
struct Part {
    static constexpr int kPer = kVec ? 16 / sizeof(T) : 1;
    uint32_t w[kVec ? 4 : 1];
    // zeros behind the row's end. Vectors by predicated loads, so that all of a thread's are on their way at once (8192 x 7168: 28.4 us, 29.5 as
    // branches)
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t cols) {
        if constexpr (kVec) {
            asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                : "l"(row + c), "r"((int)(c < cols)));
        } else if (c >= cols) {
            w[0] = 0;
        } else if constexpr (sizeof(T) == 2) {
            w[0] = (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row + c)) << 16;
        } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + c));
        }
    }
    __device__ __forceinline__ uint32_t bits(int i) const {  // of value i in fp32; i known when compiled
        if constexpr (!kVec || sizeof(T) == 4) return w[i];
        else return i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16;
    }
};

// low byte: the code
__device__ __forceinline__ uint32_t code(float x, float s, float r) {
    const float y = __fmul_rn(x, r);
    return __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-y, s, x), r, y), 12582912.0f));
}

template <typename T, bool kVec>
__device__ __forceinline__ void put(int8_t* row, int64_t c, int64_t cols, const Part<T, kVec>& v, float s, float r, bool finite) {
    if (c >= cols) return;
    if constexpr (kVec) {
        constexpr int kWords = Part<T, kVec>::kPer / 4;
        uint32_t word[kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = code(__uint_as_float(v.bits(4 * j + i)), s, r);
            word[j] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            if (!finite) word[j] = 0;
        }
        if constexpr (kWords == 1) *reinterpret_cast<uint32_t*>(row + c) = word[0];
        else *reinterpret_cast<uint2*>(row + c) = make_uint2(word[0], word[1]);
    } else {
        row[c] = finite ? (int8_t)code(__uint_as_float(v.bits(0)), s, r) : 0;
    }
}

constexpr int kShortThreads = 128;

// kHold: parts of a thread at most (all of them in registers); 0: rows of any length, read twice
template <typename T, bool kVec, int kHold, int kThreads>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t cols, int64_t x_stride, int8_t* __restrict__ q, int64_t q_stride,
                    float* __restrict__ scale, int64_t rows) {
    using P = Part<T, kVec>;
    constexpr int kStep = kThreads * P::kPer;
    __shared__ uint32_t best[2][kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
        const T* src = x + r * x_stride;
        int8_t* dst = q + r * q_stride;
        const int64_t c0 = threadIdx.x * P::kPer;
        // the largest magnitude as an integer: infinities and NaNs are above every number and survive
        uint32_t top = 0;
        auto look = [&](const P& v) {
#pragma unroll
            for (int i = 0; i < P::kPer; ++i) top = max(top, v.bits(i) & 0x7fffffffu);
        };
        P v[kHold > 0 ? kHold : 1];
        if constexpr (kHold > 0) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) v[h].load(src, c0 + h * kStep, cols);
#pragma unroll
            for (int h = 0; h < kHold; ++h) look(v[h]);
        } else {
            for (int64_t c = c0; c < cols; c += kStep) {
                v[0].load(src, c, cols);
                look(v[0]);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) best[turn][warp] = top;
        __syncthreads();  // (two sets of words in turn: the next row's are written before every warp has read these)
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) top = max(top, best[turn][w]);
        float s = __fmul_rn(__uint_as_float(top), 1.0f / 127.0f);
        if (s < 1e-8f) s = 1e-8f;
        const bool finite = s < INFINITY;
        const float inv = __fdiv_rn(1.0f, s);
        if (threadIdx.x == 0) scale[r] = s;
        if constexpr (kHold > 0) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) put(dst, c0 + h * kStep, cols, v[h], s, inv, finite);
        } else {
            for (int64_t c = c0; c < cols; c += kStep) {
                v[0].load(src, c, cols);
                put(dst, c, cols, v[0], s, inv, finite);
            }
        }
    }
}

// Short rows: L lanes have kRows of them at a time, so that their loads are on their way together.
template <typename T, bool kVec, int kHold, int L, int kRows>
__global__ void __launch_bounds__(kShortThreads)
    quantize_short_kernel(const T* __restrict__ x, int cols, int64_t x_stride, int8_t* __restrict__ q, int64_t q_stride,
                          float* __restrict__ scale, int64_t rows) {
    using P = Part<T, kVec>;
    constexpr int kGroups = kShortThreads / L;
    const int at = threadIdx.x % L, c0 = at * P::kPer;
    for (int64_t base = (int64_t)blockIdx.x * kGroups * kRows; base < rows; base += (int64_t)gridDim.x * kGroups * kRows) {
        const int64_t first = base + threadIdx.x / L;
        P v[kRows][kHold];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = first + i * kGroups;
#pragma unroll
            for (int h = 0; h < kHold; ++h) v[i][h].load(x + r * x_stride, c0 + h * L * P::kPer, r < rows ? cols : 0);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = first + i * kGroups;
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < kHold; ++h)
#pragma unroll
                for (int j = 0; j < P::kPer; ++j) top = max(top, v[i][h].bits(j) & 0x7fffffffu);
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            float s = __fmul_rn(__uint_as_float(top), 1.0f / 127.0f);
            if (s < 1e-8f) s = 1e-8f;
            const bool finite = s < INFINITY;
            const float inv = __fdiv_rn(1.0f, s);
            if (at == 0 && r < rows) scale[r] = s;
#pragma unroll
            for (int h = 0; h < kHold; ++h) put(q + r * q_stride, c0 + h * L * P::kPer, r < rows ? cols : 0, v[i][h], s, inv, finite);
        }
    }
}

template <typename T>
cudaError_t launch(const T* x, int64_t rows, int64_t cols, int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                   cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(rows, 0x7fffffff);
    constexpr int kPer = 16 / sizeof(T);
    // 16 bytes of x and as many codes at a time where every row starts on such vectors and has whole ones
    const bool vec = !((reinterpret_cast<uintptr_t>(x) | (uint64_t)(x_stride * (int64_t)sizeof(T))) & 15) &&
                     !((reinterpret_cast<uintptr_t>(q) | (uint64_t)q_stride | (uint64_t)cols) & (kPer - 1));
    // 128 threads a row (8192 x 7168 bf16 28.4 us, 32.8 with 256 and 30.6 with 64; 8192 x 1536 9.9, 12.3 and 8.7), 256 of the longest (700 x 20000
    // 11.5 us, 14.1 read twice and 19.4 held by 128)
    const int64_t parts = (cols + 128 * (vec ? kPer : 1) - 1) / (128 * (vec ? kPer : 1));
#define MOE_QUANT(vec, hold, threads) \
    quantize_kernel<T, vec, hold, threads><<<grid, threads, 0, s>>>(x, cols, x_stride, q, q_stride, scale, rows)
#define MOE_QUANT_SHORT(vec, hold, lanes, per_lane)                                                                                  \
    quantize_short_kernel<T, vec, hold, lanes, per_lane>                                                                             \
        <<<(unsigned)std::min<int64_t>((rows + kShortThreads / lanes * per_lane - 1) / (kShortThreads / lanes * per_lane), 0x7fffffff), \
           kShortThreads, 0, s>>>(x, (int)cols, x_stride, q, q_stride, scale, rows)
    // Short rows, where there are more of them than the SMs' first CTAs: lanes share a warp (bf16, CTAs of a row and lanes: 2^20 x 64 683 and 41 us,
    // 2^18 x 256 174 and 42, 65536 x 1024 57 and 33, 8192 x 256 7.3 and 3.2, 1216 x 256 2.1 and 1.7, but 152 x 256 1.5 and 1.7). Eight vectors or
    // sixteen values a lane from 32 rows an SM on (32768 x 2048 37 and 33, 8192 x 2048 10.4 and 9.8, 1216 x 2048 3.2 and 3.5).
    const int64_t per_sm = rows / tc_num_sms(), unit = vec ? kPer : 2;
    if (per_sm >= (cols <= 128 * unit ? 4 : 32) && cols <= 256 * unit) {
        const int64_t units = (cols + unit - 1) / unit;
        if (vec) {
            if (units <= 4) MOE_QUANT_SHORT(true, 1, 4, 2);
            else if (units <= 8) MOE_QUANT_SHORT(true, 1, 8, 2);
            else if (units <= 16) MOE_QUANT_SHORT(true, 1, 16, 2);
            else if (units <= 32) MOE_QUANT_SHORT(true, 1, 32, 2);
            else if (units <= 64) MOE_QUANT_SHORT(true, 2, 32, 2);
            else if (units <= 128) MOE_QUANT_SHORT(true, 4, 32, 1);
            else MOE_QUANT_SHORT(true, 8, 32, 1);
        } else if (units <= 32) MOE_QUANT_SHORT(false, 2, 32, 4);
        else if (units <= 64) MOE_QUANT_SHORT(false, 4, 32, 2);
        else if (units <= 128) MOE_QUANT_SHORT(false, 8, 32, 1);
        else MOE_QUANT_SHORT(false, 16, 32, 1);
    } else if (vec) {
        if (parts <= 2) MOE_QUANT(true, 2, 128);
        else if (parts <= 4) MOE_QUANT(true, 4, 128);
        else if (parts <= 8) MOE_QUANT(true, 8, 128);
        else if (parts <= 16) MOE_QUANT(true, 16, 128);
        else if (parts <= 32) MOE_QUANT(true, 16, 256);
        else MOE_QUANT(true, 0, 256);
    } else {
        // single values: rows of up to 1024 held; longer ones are read twice (8192 x 701 bf16 8.8 us held and 10.3, 8192 x 3001 33 and 25)
        if (parts <= 8) MOE_QUANT(false, 8, 128);
        else if (parts <= 128) MOE_QUANT(false, 0, 128);
        else MOE_QUANT(false, 0, 256);
    }
#undef MOE_QUANT
#undef MOE_QUANT_SHORT
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
