// The rows of a token's experts back to the token, weighted, and the gradients (moe_unpermute, moe_unpermute_backward in moe_ops.h).
//
// Bound by HBM: every row is read once (and its gradient written). Forward: a warp has a segment of a token's columns and
// adds the K rows in the order of k, eight loads on their way a lane. Backward: a group of warps has a slot; it reads the row and the
// token's gradient (which the token's other slots find in cache), writes the row's gradient and adds up their product.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// N consecutive elements of T: one vector where they are 16 bytes (or two, fp32 opposite bf16), else one by one
template <typename T, int N>
__device__ __forceinline__ void load(const T* p, float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) v[0] = bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(p)));
        else v[0] = __ldg(reinterpret_cast<const float*>(p));
    } else if constexpr (sizeof(T) == 2) {
        static_assert(N == 8, "one vector");
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(p) + j);
            v[4 * j] = w.x, v[4 * j + 1] = w.y, v[4 * j + 2] = w.z, v[4 * j + 3] = w.w;
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint16_t*>(p) = float_to_bf16_bits(v[0]);
        else *reinterpret_cast<float*>(p) = v[0];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = (uint32_t)float_to_bf16_bits(v[2 * j]) | ((uint32_t)float_to_bf16_bits(v[2 * j + 1]) << 16);
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
            reinterpret_cast<float4*>(p)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
}

// row of slot `lane` of a token, or -1
__device__ __forceinline__ int slot_row_of(const UnpermuteArgs& p, int64_t slot, bool there) {
    const int r = there ? __ldg(p.slot_row + slot) : -1;
    return r >= 0 && r < p.T * p.K ? r : -1;
}

template <typename R, typename Y, int N>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(UnpermuteArgs p, int64_t segments) {
    const int lane = threadIdx.x & 31;
    const int64_t items = p.T * segments;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < items; item += (int64_t)gridDim.x * kWarps) {
        const int64_t t = item / segments, c = (item - t * segments) * (32 * N) + lane * N;
        const int my_row = slot_row_of(p, t * p.K + lane, lane < p.K);
        const float my_w = p.weights && my_row >= 0 ? __ldg(p.weights + t * p.K + lane) : 1.0f;
        const R* rows = static_cast<const R*>(p.rows);
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        constexpr int kBatch = 8;  // rows on their way
        for (int k0 = 0; k0 < p.K; k0 += kBatch) {
            float v[kBatch][N], w[kBatch];
            int r[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                r[b] = __shfl_sync(0xffffffffu, my_row, (k0 + b) & 31);
                w[b] = __shfl_sync(0xffffffffu, my_w, (k0 + b) & 31);
                if (k0 + b >= p.K) r[b] = -1;
                if (r[b] >= 0 && c < p.H) load<R, N>(rows + (int64_t)r[b] * p.rows_stride + c, v[b]);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (r[b] >= 0 && c < p.H)
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = __fmaf_rn(w[b], v[b][j], acc[j]);
        }
        if (c < p.H) store<Y, N>(static_cast<Y*>(p.out) + t * p.out_stride + c, acc);
    }
}

// G warps a slot
template <typename R, typename Y, int N, int G>
__global__ void __launch_bounds__(kThreads) backward_kernel(UnpermuteArgs p) {
    __shared__ float part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % G;
    const int64_t slot = (int64_t)blockIdx.x * (kWarps / G) + warp / G, slots = (int64_t)p.T * p.K;
    const int row = slot_row_of(p, slot, slot < slots);
    float dot = 0.0f;
    if (row >= 0) {
        const float w = p.weights ? __ldg(p.weights + slot) : 1.0f;
        const Y* dy = static_cast<const Y*>(p.dy) + slot / p.K * p.dy_stride;
        const R* in = static_cast<const R*>(p.rows) + (int64_t)row * p.rows_stride;
        R* out = static_cast<R*>(p.out) + (int64_t)row * p.out_stride;
        constexpr int kBatch = 4;
        for (int64_t c0 = (int64_t)sub * 32 * N * kBatch; c0 < p.H; c0 += (int64_t)G * 32 * N * kBatch) {
            float a[kBatch][N], b[kBatch][N];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t c = c0 + (j * 32 + lane) * N;
                if (c < p.H) {
                    load<Y, N>(dy + c, a[j]);
                    if (p.d_weights) load<R, N>(in + c, b[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t c = c0 + (j * 32 + lane) * N;
                if (c >= p.H) continue;
                if (p.d_weights)
#pragma unroll
                    for (int i = 0; i < N; ++i) dot = __fmaf_rn(a[j][i], b[j][i], dot);
#pragma unroll
                for (int i = 0; i < N; ++i) a[j][i] *= w;
                store<R, N>(out + c, a[j]);
            }
        }
    }
    if (!p.d_weights) return;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if constexpr (G > 1) {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        dot = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) dot += part[warp / G * G + g];
    }
    if (sub == 0 && lane == 0 && slot < slots) p.d_weights[slot] = dot;
}

template <typename R, typename Y, int N>
cudaError_t launch_forward(const UnpermuteArgs& a, cudaStream_t s) {
    const int64_t segments = (a.H + 32 * N - 1) / (32 * N), ctas = (a.T * segments + kWarps - 1) / kWarps;
    unpermute_kernel<R, Y, N><<<(unsigned)std::min<int64_t>(ctas, 0x7fffffff), kThreads, 0, s>>>(a, segments);
    return cudaGetLastError();
}

template <typename R, typename Y, int N>
cudaError_t launch_back(const UnpermuteArgs& a, cudaStream_t s) {
    const int64_t slots = (int64_t)a.T * a.K;
    // a CTA a slot while the slots do not give every SM a few CTAs of eight
    if (slots < (int64_t)tc_num_sms() * 4 * kWarps) backward_kernel<R, Y, N, kWarps><<<(unsigned)slots, kThreads, 0, s>>>(a);
    else backward_kernel<R, Y, N, 1><<<(unsigned)((slots + kWarps - 1) / kWarps), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// eight columns at a time where every row of either matrix starts on 16 bytes and has a multiple of eight
bool vectors(const UnpermuteArgs& a) {
    const uint64_t r = a.type == MOE_TYPE_BF16 ? 2 : 4, t = a.token_type == MOE_TYPE_BF16 ? 2 : 4;
    const bool back = a.dy != nullptr;
    uint64_t low = reinterpret_cast<uintptr_t>(a.rows) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.out);
    low |= (uint64_t)a.out_stride * (back ? r : t);
    if (a.rows) low |= (uint64_t)a.rows_stride * r;
    if (back) low |= (uint64_t)a.dy_stride * t;
    return low % 16 == 0 && a.H % 8 == 0;
}

template <bool kBack, typename R, typename Y>
cudaError_t launch_ry(const UnpermuteArgs& a, cudaStream_t s) {
    if constexpr (kBack) return vectors(a) ? launch_back<R, Y, 8>(a, s) : launch_back<R, Y, 1>(a, s);
    else return vectors(a) ? launch_forward<R, Y, 8>(a, s) : launch_forward<R, Y, 1>(a, s);
}

template <bool kBack>
cudaError_t launch_any(const UnpermuteArgs& a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (a.type == MOE_TYPE_BF16)
        return a.token_type == MOE_TYPE_BF16 ? launch_ry<kBack, __nv_bfloat16, __nv_bfloat16>(a, s)
                                             : launch_ry<kBack, __nv_bfloat16, float>(a, s);
    return a.token_type == MOE_TYPE_BF16 ? launch_ry<kBack, float, __nv_bfloat16>(a, s) : launch_ry<kBack, float, float>(a, s);
}

}  // namespace

cudaError_t launch_unpermute(const UnpermuteArgs& a, cudaStream_t s) { return launch_any<false>(a, s); }
cudaError_t launch_unpermute_backward(const UnpermuteArgs& a, cudaStream_t s) { return launch_any<true>(a, s); }

}  // namespace moe
