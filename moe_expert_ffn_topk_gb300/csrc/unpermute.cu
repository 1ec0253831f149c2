// The rows of a token's experts back to the token, weighted, and the gradients (moe_unpermute, moe_unpermute_backward in moe_ops.h).
//
// Bound by HBM: every row is read once (and its gradient written). Forward: a warp has a segment of a token's columns and
// adds the K rows in the order of k, eight loads on their way a lane (of several segments where K is small). Backward: a group of warps has a slot; it reads the row and the
// token's gradient (which the token's other slots find in cache), writes the row's gradient and adds up their product.
// Measured: forward 8192 x 8 x 7168 bf16 (1.06 GB) 167 us, 0.95 of the copy rate (281 with one load on its way at a time); backward 16384 x
// 2 x 4096 bf16 (0.67 GB) 99 us, the copy rate; 333 x 6 x 1531 fp32 (27 MB, single columns) 8.0 us, 0.49, a wave of short runs of loads.
// 7 x 8 x 7168 forward: 2.4 us on the device.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch1 = 8, kBatchN = 4;  // loads of a lane on their way in the backward pass, of single columns and of vectors

// N consecutive elements of T as they lie in memory: a lane holds these while its loads are on their way
template <typename T, int N>
struct Packed {
    static constexpr int kBytes = N * (int)sizeof(T);
    static_assert(N == 1 || kBytes % 8 == 0, "whole vectors");
    uint32_t w[kBytes < 4 ? 1 : kBytes / 4];

    // zeros where `on` is false. Predicated loads, not branches: the compiler joined a branch around a load with that around its
    // use, and a warp had one load on its way instead of eight
    __device__ __forceinline__ void load(const T* p, bool on) {
        if constexpr (kBytes == 2) {
            uint16_t v;
            asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}" : "=h"(v) : "l"(p), "r"((int)on));
            w[0] = v;
        } else if constexpr (kBytes == 4) {
            asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}" : "=r"(w[0]) : "l"(p), "r"((int)on));
        } else if constexpr (kBytes == 8) {
            asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t@p ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
                : "=r"(w[0]), "=r"(w[1])
                : "l"(p), "r"((int)on));
        } else {
#pragma unroll
            for (int j = 0; j < kBytes / 16; ++j)
                asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                    "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                    : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                    : "l"(reinterpret_cast<const uint4*>(p) + j), "r"((int)on));
        }
    }
    __device__ __forceinline__ float at(int i) const {  // i known when compiled
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

template <typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&v)[N]) {
    if constexpr (N == 1 && sizeof(T) == 2) *reinterpret_cast<uint16_t*>(p) = float_to_bf16_bits(v[0]);
    else if constexpr (N == 1) *reinterpret_cast<float*>(p) = v[0];
    else if constexpr (sizeof(T) == 2) {
        uint32_t u[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) u[j] = (uint32_t)float_to_bf16_bits(v[2 * j]) | ((uint32_t)float_to_bf16_bits(v[2 * j + 1]) << 16);
        if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
        else *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
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

// S segments of 8 / S rows are on their way at a time (S > 1: of all the token's rows).
// A warp's item is a token's run of `per` segments of 32 * N columns; the next item's slots and weights are on their way while one is
// worked on (an item's own are a load that its rows' loads wait for).
template <typename R, typename Y, int N, int S>
__global__ void __launch_bounds__(kThreads, 3) unpermute_kernel(UnpermuteArgs p, int64_t parts, int64_t per) {
    const int lane = threadIdx.x & 31;
    const int64_t items = p.T * parts, step = (int64_t)gridDim.x * kWarps;
    int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const R* rows = static_cast<const R*>(p.rows);
    int next_row = -1;
    float next_w = 0.0f;
    auto fetch = [&](int64_t i) {
        const int64_t slot = i / parts * p.K + lane;
        const bool there = i < items && lane < p.K;
        next_row = slot_row_of(p, slot, there);
        next_w = p.weights && there ? __ldg(p.weights + slot) : 1.0f;
    };
    fetch(item);
    for (; item < items; item += step) {
        const int64_t t = item / parts, c0 = (item - t * parts) * per * (32 * N);
        const int my_row = next_row;
        const float my_w = my_row >= 0 ? next_w : 0.0f;
        fetch(item + step);
        const int64_t c1 = min(p.H, c0 + per * (32 * N));
        for (int64_t c = c0 + lane * N; c - lane * N < c1; c += S * 32 * N) {
            constexpr int kBatch = 8 / S;  // rows on their way
            Packed<R, N> v[S][kBatch];
            auto load = [&](int k0) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int r = __shfl_sync(0xffffffffu, my_row, (k0 + b) & 31);
#pragma unroll
                    for (int i = 0; i < S; ++i) {
                        const int64_t at = c + i * 32 * N;
                        v[i][b].load(rows + (int64_t)r * p.rows_stride + at, r >= 0 && k0 + b < p.K && at < c1);
                    }
                }
            };
            auto add = [&](int k0, int i, float (&acc)[N]) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {  // (a slot without a row: 0 * 0)
                    const float w = __shfl_sync(0xffffffffu, my_w, (k0 + b) & 31);
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = __fmaf_rn(w, v[i][b].at(j), acc[j]);
                }
            };
            if constexpr (S > 1) load(0);  // (all of the token's rows)
#pragma unroll
            for (int i = 0; i < S; ++i) {
                float acc[N];
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = 0.0f;
                if constexpr (S > 1) {
                    add(0, i, acc);
                } else {
                    for (int k0 = 0; k0 < p.K; k0 += kBatch) {
                        load(k0);
                        add(k0, 0, acc);
                    }
                }
                const int64_t at = c + i * 32 * N;
                if (at < c1) store<Y, N>(static_cast<Y*>(p.out) + t * p.out_stride + at, acc);
            }
        }
    }
}

// G warps a slot
template <typename R, typename Y, int N, int G>
__global__ void __launch_bounds__(kThreads) backward_kernel(UnpermuteArgs p) {
    __shared__ float part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % G;
    const int64_t slot = (int64_t)blockIdx.x * (kWarps / G) + warp / G, slots = (int64_t)p.T * p.K;
    const bool there = slot < slots;
    const float w = p.weights && there ? __ldg(p.weights + slot) : 1.0f;
    const int row = slot_row_of(p, slot, there);
    const Y* dy = static_cast<const Y*>(p.dy) + (there ? slot / p.K : 0) * p.dy_stride;
    const R* in = static_cast<const R*>(p.rows) + (int64_t)row * p.rows_stride;
    R* out = static_cast<R*>(p.out) + (int64_t)row * p.out_stride;
    float dot = 0.0f;
    constexpr int kBatch = N == 1 ? kBatch1 : kBatchN;
    for (int64_t c0 = (int64_t)sub * 32 * N * kBatch; c0 < p.H; c0 += (int64_t)G * 32 * N * kBatch) {
        Packed<Y, N> a[kBatch];
        Packed<R, N> b[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {  // (the token's values first: they do not wait for the slot's row)
            const int64_t c = c0 + (j * 32 + lane) * N;
            a[j].load(dy + c, there && c < p.H);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t c = c0 + (j * 32 + lane) * N;
            b[j].load(in + c, p.d_weights && row >= 0 && c < p.H);
        }
        if (row < 0) break;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t c = c0 + (j * 32 + lane) * N;
            if (c >= p.H) continue;
            if (p.d_weights)
#pragma unroll
                for (int i = 0; i < N; ++i) dot = __fmaf_rn(a[j].at(i), b[j].at(i), dot);
            float grad[N];
#pragma unroll
            for (int i = 0; i < N; ++i) grad[i] = a[j].at(i) * w;
            store<R, N>(out + c, grad);
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

// Q slots a warp, of rows that fit in a Q-th of its loads
template <typename R, typename Y, int N, int Q>
__global__ void __launch_bounds__(kThreads) backward_short_kernel(UnpermuteArgs p) {
    constexpr int kBatch = (N == 1 ? kBatch1 : kBatchN) / Q;
    const int lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * Q, slots = (int64_t)p.T * p.K;
    int row[Q];
    float w[Q];
    Packed<Y, N> a[Q][kBatch];
    Packed<R, N> b[Q][kBatch];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const bool there = first + i < slots;
        row[i] = slot_row_of(p, first + i, there);
        w[i] = p.weights && there ? __ldg(p.weights + first + i) : 1.0f;
        const Y* dy = static_cast<const Y*>(p.dy) + (there ? (first + i) / p.K : 0) * p.dy_stride;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t c = (j * 32 + lane) * N;
            a[i][j].load(dy + c, there && c < p.H);
        }
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const R* in = static_cast<const R*>(p.rows) + (int64_t)row[i] * p.rows_stride;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t c = (j * 32 + lane) * N;
            b[i][j].load(in + c, p.d_weights && row[i] >= 0 && c < p.H);
        }
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        R* out = static_cast<R*>(p.out) + (int64_t)row[i] * p.out_stride;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t c = (j * 32 + lane) * N;
            if (row[i] < 0 || c >= p.H) continue;
            float grad[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                dot = __fmaf_rn(a[i][j].at(e), b[i][j].at(e), dot);
                grad[e] = a[i][j].at(e) * w[i];
            }
            store<R, N>(out + c, grad);
        }
        if (!p.d_weights) continue;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0 && first + i < slots) p.d_weights[first + i] = dot;
    }
}

template <typename R, typename Y, int N, int S>
cudaError_t launch_segments(const UnpermuteArgs& a, int64_t segments, int64_t resident, cudaStream_t s) {
    // longer runs a warp where that leaves every resident warp several items
    int64_t per = S;
    while (per < 4 && per * 2 <= segments && a.T * ((segments + 2 * per - 1) / (2 * per)) >= 8 * resident) per *= 2;
    const int64_t parts = (segments + per - 1) / per, ctas = (a.T * parts + kWarps - 1) / kWarps;
    unpermute_kernel<R, Y, N, S><<<(unsigned)std::min<int64_t>(ctas, resident / kWarps), kThreads, 0, s>>>(a, parts, per);
    return cudaGetLastError();
}

template <typename R, typename Y, int N>
cudaError_t launch_forward(const UnpermuteArgs& a, cudaStream_t s) {
    const int64_t segments = (a.H + 32 * N - 1) / (32 * N), resident = (int64_t)tc_num_sms() * 3 * kWarps;
    // A token of few rows: several segments at a time, where every resident warp has an item all the same (bf16, one and several: 16384 x 2 x 4096
    // 115 and 65 us, 1024 x 2 x 4096 10.2 and 5.0, 16384 x 2 x 2047 279 and 116, 16384 x 4 x 2048 64.5 and 55.4).
    if (a.K <= 2 && segments >= 4 && a.T * (segments / 4) >= resident) return launch_segments<R, Y, N, 4>(a, segments, resident, s);
    if (a.K <= 4 && segments >= 2 && a.T * (segments / 2) >= resident) return launch_segments<R, Y, N, 2>(a, segments, resident, s);
    return launch_segments<R, Y, N, 1>(a, segments, resident, s);
}

template <typename R, typename Y, int N>
cudaError_t launch_back(const UnpermuteArgs& a, cudaStream_t s) {
    const int64_t slots = (int64_t)a.T * a.K, part = 32 * N * (N == 1 ? kBatch1 : kBatchN);
    // warps a slot: no more than its row has parts for (4096 slots of 512 bf16: 3.3 us with one, 9.8 with eight), doubled while the SMs hold them
    // all, 48 each (bf16, H 4096: 512 slots 2.9 us with four and 4.8 with one, 2048 slots 8.0 with two, 9.6 with one, 11.6 with eight)
    int G = 1;
    while (G < kWarps && (a.H + part - 1) / part > G && slots * G * 2 <= (int64_t)tc_num_sms() * 48) G *= 2;
    // short rows: several slots a warp, where every resident warp has some all the same (bf16, one and several: 32768 x 8 x 256 114 and 57 us,
    // 4096 x 8 x 256 13.8 and 8.6, 16384 x 8 x 512 69 and 50, 16384 x 8 x 63 52 and 19)
    if (G == 1) {
        const int64_t resident = (int64_t)tc_num_sms() * 48;
        if (a.H <= part / 4 && slots >= resident * 4) {
            backward_short_kernel<R, Y, N, 4><<<(unsigned)((slots + 4 * kWarps - 1) / (4 * kWarps)), kThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        if (a.H <= part / 2 && slots >= resident * 2) {
            backward_short_kernel<R, Y, N, 2><<<(unsigned)((slots + 2 * kWarps - 1) / (2 * kWarps)), kThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
    }
    const unsigned ctas = (unsigned)((slots * G + kWarps - 1) / kWarps);
    if (G == 1) backward_kernel<R, Y, N, 1><<<ctas, kThreads, 0, s>>>(a);
    else if (G == 2) backward_kernel<R, Y, N, 2><<<ctas, kThreads, 0, s>>>(a);
    else if (G == 4) backward_kernel<R, Y, N, 4><<<ctas, kThreads, 0, s>>>(a);
    else backward_kernel<R, Y, N, 8><<<ctas, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// 16 bytes of a row at a time where every row of either matrix starts on 16 bytes and has whole vectors of the experts' rows
bool vectors(const UnpermuteArgs& a) {
    const uint64_t r = a.type == MOE_TYPE_BF16 ? 2 : 4, t = a.token_type == MOE_TYPE_BF16 ? 2 : 4;
    const bool back = a.dy != nullptr;
    uint64_t low = reinterpret_cast<uintptr_t>(a.rows) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.out);
    low |= (uint64_t)a.out_stride * (back ? r : t);
    if (a.rows) low |= (uint64_t)a.rows_stride * r;
    if (back) low |= (uint64_t)a.dy_stride * t;
    return low % 16 == 0 && a.H % (int64_t)(16 / r) == 0;
}

template <bool kBack, typename R, typename Y>
cudaError_t launch_ry(const UnpermuteArgs& a, cudaStream_t s) {
    if constexpr (kBack) return vectors(a) ? launch_back<R, Y, 16 / sizeof(R)>(a, s) : launch_back<R, Y, 1>(a, s);
    else return vectors(a) ? launch_forward<R, Y, 16 / sizeof(R)>(a, s) : launch_forward<R, Y, 1>(a, s);
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
