// Product of e4m3 matrices with fp32 scales for each block of 128 (moe_fp8_matmul in moe_ops.h).
#include "common.cuh"
#include "ops.h"

namespace moe {

namespace {

constexpr int kTile = 64, kBK = 32;

struct Args {
    moe_fp8_matmul_args a;
    int kb_count, nb_count;
};

// One 64 x 64 tile of one group per CTA: fp32 products and sums on the CUDA cores, one partial sum a block of K.
template <typename Out>
__global__ void __launch_bounds__(256) simple_kernel(Args p) {
    __shared__ float sa[kTile][kBK + 1], sb[kTile][kBK + 1];
    const int g = blockIdx.z;
    int64_t lo = 0, hi = p.a.M;
    if (p.a.offsets) {
        lo = min(max((int64_t)p.a.offsets[g], (int64_t)0), p.a.M);
        hi = min(max((int64_t)p.a.offsets[g + 1], (int64_t)0), p.a.M);
    }
    const int n0 = blockIdx.x * kTile;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const uint8_t* b = static_cast<const uint8_t*>(p.a.b) + (int64_t)g * p.a.N * p.a.b_stride;
    const float* bs = p.a.b_scale + (int64_t)g * p.nb_count * p.kb_count;
    for (int64_t m0 = lo + (int64_t)blockIdx.y * kTile; m0 < hi; m0 += (int64_t)gridDim.y * kTile) {
        float acc[4][4] = {};
        for (int kb = 0; kb < p.kb_count; ++kb) {
            float part[4][4] = {};
            for (int k0 = kb * 128; k0 < min((int64_t)(kb + 1) * 128, p.a.K); k0 += kBK) {
                __syncthreads();
                for (int i = threadIdx.x; i < kTile * kBK; i += 256) {
                    const int r = i / kBK, c = i % kBK;
                    const bool in = k0 + c < p.a.K;
                    sa[r][c] = in && m0 + r < hi
                                   ? e4m3_to_float(static_cast<const uint8_t*>(p.a.a)[(m0 + r) * p.a.a_stride + k0 + c])
                                   : 0.0f;
                    sb[r][c] = in && n0 + r < p.a.N ? e4m3_to_float(b[(int64_t)(n0 + r) * p.a.b_stride + k0 + c]) : 0.0f;
                }
                __syncthreads();
                for (int c = 0; c < kBK; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[ty + 16 * i][c], sb[tx + 16 * j][c], part[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty + 16 * i;
                if (m >= hi) continue;
                const float s = p.a.a_scale[m * p.kb_count + kb];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + tx + 16 * j;
                    if (n < p.a.N) acc[i][j] = fmaf(part[i][j], s * bs[(int64_t)(n / 128) * p.kb_count + kb], acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i;
                const int n = n0 + tx + 16 * j;
                if (m < hi && n < p.a.N) static_cast<Out*>(p.a.out)[m * p.a.out_stride + n] = Out(acc[i][j]);
            }
    }
}

}  // namespace

size_t fp8_matmul_workspace(int64_t, int64_t, int64_t, int) { return 256; }

cudaError_t launch_fp8_matmul(const moe_fp8_matmul_args& a, void*, cudaStream_t s) {
    if (a.M == 0) return cudaSuccess;
    Args p{a, (int)((a.K + 127) / 128), (int)((a.N + 127) / 128)};
    const int64_t rows = (a.M + kTile - 1) / kTile;
    const dim3 grid((unsigned)((a.N + kTile - 1) / kTile), (unsigned)(rows < 1024 ? rows : 1024), (unsigned)a.groups);
    if (a.out_type == MOE_TYPE_BF16) simple_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else simple_kernel<float><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace moe
