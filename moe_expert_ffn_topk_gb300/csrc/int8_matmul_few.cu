// moe_int8_matmul (moe_ops.h) for a few rows a group: bound by reading the weights once. A CTA has 16 weight rows and its eight warps a part
// of K each (with few weight rows, so have the CTAs of a cluster); a lane reads 32 bytes of a weight row at a time, straight to
// the registers that mma.sync m16n8k32 on int8 takes (the order of K within a row's 128 codes is the same for both operands, so
// it need not be the instruction's), eight tokens a time. The sums are integers, so their order does not matter.
//
// mma.sync on int8 runs at 150 TOP/s, dp4a too: eight rows of a take 0.7 of the time there that their weights' bytes take from HBM, sixteen 1.4. Up to
// four are multiplied by dp4a, which does no work for rows that are not there. Measured on 4096 x 7168 (29 MB, 4.4 us at the copy rate; graph
// of calls, inputs rotated past L2): 1 row 7.4-7.7 us, 4 rows 9.0-9.3, 8 rows 9.6, 16 rows 12.9 (1 row by mma.sync 9.1). What is left is start,
// two steps of loads in flight a warp, and the sum: a third and a fourth step spilled and gained nothing.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "int8_matmul.h"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStepK = 128;
constexpr int kMaxSplit = 8;  // CTAs of a cluster

struct FewArgs {
    const int8_t* a;
    const int8_t* b;
    const float* a_scale;
    const float* b_scale;
    const int32_t* offsets;
    void* out;
    int64_t a_stride, b_stride, out_stride;
    int M, N, K, groups, split;  // split: CTAs of a cluster that share K
};

// 32 bytes, or zeros
__device__ __forceinline__ void load32(uint32_t (&v)[8], const int8_t* p, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %9, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
        : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void load16(uint32_t* v, const int8_t* p, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "l"(p), "r"((int)on));
}

// c += 16 weight rows (two of a lane: words of u and v) x 8 tokens (words of t)
__device__ __forceinline__ void mma8(int (&c)[4], uint32_t u0, uint32_t v0, uint32_t u1, uint32_t v1, uint32_t t0, uint32_t t1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(u0), "r"(v0), "r"(u1), "r"(v1), "r"(t0), "r"(t1));
}

// kTokens: tokens that a pass over the weights serves; 8 or 16 by mma.sync, up to 4 by dp4a (a lane multiplies its bytes of the two rows with
// those of every token). kWide: rows of a and b start on 32 bytes and K is a multiple of 32, so that a
// lane loads 32 bytes at a time (the four lanes of a row 128), else twice 16
template <int kTokens, bool kWide, typename Out>
__global__ void __launch_bounds__(kThreads, kTokens <= 2 || kTokens == 8 ? 3 : 2) few_kernel(FewArgs p) {
    constexpr bool kMma = kTokens >= 8;
    constexpr int kTiles = kMma ? kTokens / 8 : kTokens;  // rows of a that a lane reads
    __shared__ int sums[kWarps][kTokens][16];
    __shared__ int bounds[2], total[kTokens * 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.y, n0 = (int)(blockIdx.x / p.split) * 16;
    const uint32_t rank = p.split > 1 ? cluster_ctarank() : 0u;
    int lo = 0, hi = p.M;
    if (p.offsets) {
        // offsets are taken into [0, M], and one below an earlier one as that one
        if (warp == 0) {
            int last = 0;
            for (int j = lane; j <= g; j += 32) last = max(last, min(__ldg(p.offsets + j), p.M));
            last = __reduce_max_sync(0xffffffffu, last);
            if (lane == 0) bounds[0] = last, bounds[1] = max(last, min(__ldg(p.offsets + g + 1), p.M));
        }
        __syncthreads();
        lo = bounds[0], hi = bounds[1];
    }
    if (lo >= hi) return;  // (every CTA of the cluster)
    // this warp's part of K, whole steps
    const int parts = p.split * kWarps, part = (int)rank * kWarps + warp, steps = (p.K + kStepK - 1) / kStepK;
    const int k0 = (int)((int64_t)steps * part / parts) * kStepK, k1 = (int)((int64_t)steps * (part + 1) / parts) * kStepK;
    const int r = lane >> 2, at = (lane & 3) * 32;  // rows r and r + 8 of the weights, token r; the lane's 32 bytes of 128
    const bool on0 = n0 + r < p.N, on1 = n0 + r + 8 < p.N;
    const int8_t* w0 = p.b + ((int64_t)g * p.N + n0 + r) * p.b_stride + at;
    const int8_t* w1 = w0 + 8 * p.b_stride;
    // of the value that the thread writes; on its way during the product
    const float b_scale = n0 + (int)threadIdx.x % 16 < p.N ? __ldg(p.b_scale + (int64_t)g * p.N + n0 + threadIdx.x % 16) : 0.0f;
    for (int m0 = lo; m0 < hi; m0 += kTokens) {
        int c[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0;
        const int first = kMma ? m0 + r : m0;
        constexpr int kApart = kMma ? 8 : 1;
        const int8_t* x = p.a + (int64_t)first * p.a_stride + at;
        uint32_t u[2][8], v[2][8], t[2][kTiles][8];  // the next step's on their way while one is multiplied
        auto load = [&](int buf, int k) {
            auto row = [&](uint32_t (&d)[8], const int8_t* p8, bool on) {
                if constexpr (kWide) {
                    load32(d, p8 + k, on && k < k1 && k + at < p.K);
                } else {
                    load16(d, p8 + k, on && k < k1 && k + at < p.K);
                    load16(d + 4, p8 + k + 16, on && k < k1 && k + at + 16 < p.K);
                }
            };
            row(u[buf], w0, on0);
            row(v[buf], w1, on1);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) row(t[buf][i], x + kApart * i * p.a_stride, first + kApart * i < hi);
        };
        auto multiply = [&](int buf) {
#pragma unroll
            for (int h = 0; h < 8; h += 2)
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    if constexpr (kMma) {
                        mma8(c[i], u[buf][h], v[buf][h], u[buf][h + 1], v[buf][h + 1], t[buf][i][h], t[buf][i][h + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            c[i][2 * e] = __dp4a((int)u[buf][h + e], (int)t[buf][i][h + e], c[i][2 * e]);
                            c[i][2 * e + 1] = __dp4a((int)v[buf][h + e], (int)t[buf][i][h + e], c[i][2 * e + 1]);
                        }
                    }
                }
        };
        load(0, k0);
        for (int k = k0; k < k1; k += 2 * kStepK) {
            load(1, k + kStepK);
            multiply(0);  // (zeros behind the last step)
            load(0, k + 2 * kStepK);
            multiply(1);
        }
        // sums[warp][token][weight row]
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            if constexpr (kMma) {  // lane (r, q) holds rows r, r + 8 of tokens 2q, 2q + 1
#pragma unroll
                for (int j = 0; j < 4; ++j) sums[warp][8 * i + (lane & 3) * 2 + (j & 1)][r + 8 * (j >> 1)] = c[i][j];
            } else {  // the four lanes of a row hold parts of K
                int lower = c[i][0] + c[i][2], upper = c[i][1] + c[i][3];
#pragma unroll
                for (int d = 1; d < 4; d *= 2) {
                    lower += __shfl_xor_sync(0xffffffffu, lower, d);
                    upper += __shfl_xor_sync(0xffffffffu, upper, d);
                }
                if ((lane & 3) == 0) sums[warp][i][r] = lower, sums[warp][i][r + 8] = upper;
            }
        }
        __syncthreads();
        // the warps' sums, then those of the cluster's CTAs, a share of the values each
        static_assert(kTokens * 16 <= kThreads, "a value a thread");
        int sum = 0;
        if (threadIdx.x < kTokens * 16)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += (&sums[w][0][0])[threadIdx.x];
        bool mine = threadIdx.x < kTokens * 16;
        if (p.split > 1) {
            if (mine) total[threadIdx.x] = sum;
            cluster_sync();
            mine = mine && threadIdx.x % p.split == rank;
            if (mine) {
                int s[kMaxSplit];
#pragma unroll
                for (int k = 0; k < kMaxSplit; ++k) {  // (all on their way at once)
                    s[k] = 0;
                    if (k < p.split)
                        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                                     : "=r"(s[k])
                                     : "r"(mapa_shared(smem_u32(total + threadIdx.x), (uint32_t)k))
                                     : "memory");
                }
                sum = 0;
#pragma unroll
                for (int k = 0; k < kMaxSplit; ++k) sum += s[k];
            }
        }
        // nobody leaves, or writes its next sums, while these are read (before the stores, which the barrier would wait for)
        if (p.split > 1) cluster_sync();
        else __syncthreads();
        const int m = m0 + threadIdx.x / 16, n = n0 + threadIdx.x % 16;
        if (mine && m < hi && n < p.N) {
            const float y = int8_scaled((float)sum, b_scale, __ldg(p.a_scale + m));
            if constexpr (sizeof(Out) == 2) static_cast<uint16_t*>(p.out)[(int64_t)m * p.out_stride + n] = float_to_bf16_bits(y);
            else static_cast<float*>(p.out)[(int64_t)m * p.out_stride + n] = y;
        }
    }
}

template <int kTokens, bool kWide, typename Out>
cudaError_t launch(const FewArgs& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + 15) / 16 * p.split), (unsigned)p.groups);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, few_kernel<kTokens, kWide, Out>, p);
}

template <bool kWide, typename Out>
cudaError_t launch_tokens(const FewArgs& p, cudaStream_t s) {
    // of groups the rows are not known here: tiles of 16 (a group of more takes the weights from L2 again)
    const int rows = p.groups == 1 ? p.M : 16;
    if (rows <= 1) return launch<1, kWide, Out>(p, s);
    if (rows <= 2) return launch<2, kWide, Out>(p, s);
    if (rows <= 4) return launch<4, kWide, Out>(p, s);
    return rows <= 8 ? launch<8, kWide, Out>(p, s) : launch<16, kWide, Out>(p, s);
}

template <typename Out>
cudaError_t launch_out(const FewArgs& p, cudaStream_t s) {
    const bool wide = !((reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b) | (uint64_t)p.a_stride | (uint64_t)p.b_stride |
                         (uint64_t)p.K) & 31);
    return wide ? launch_tokens<true, Out>(p, s) : launch_tokens<false, Out>(p, s);
}

}  // namespace

cudaError_t launch_int8_few(const moe_int8_matmul_args& a, cudaStream_t s) {
    FewArgs p = {};
    p.a = static_cast<const int8_t*>(a.a);
    p.b = static_cast<const int8_t*>(a.b);
    p.a_scale = a.a_scale;
    p.b_scale = a.b_scale;
    p.offsets = a.offsets;
    p.out = a.out;
    p.a_stride = a.a_stride, p.b_stride = a.b_stride, p.out_stride = a.out_stride;
    p.M = (int)a.M, p.N = (int)a.N, p.K = (int)a.K, p.groups = a.groups;
    // K over a cluster's CTAs where the weight rows give every SM less than a CTA, while every warp keeps a step
    p.split = 1;
    while (p.split < kMaxSplit && (int64_t)(a.N + 15) / 16 * a.groups * p.split < tc_num_sms() && a.K >= (int64_t)kStepK * kWarps * 2 * p.split) p.split *= 2;
    return a.out_type == MOE_TYPE_BF16 ? launch_out<__nv_bfloat16>(p, s) : launch_out<float>(p, s);
}

}  // namespace moe
