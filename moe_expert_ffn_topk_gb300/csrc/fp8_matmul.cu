// Product of e4m3 matrices with fp32 scales for each block of 128 (moe_fp8_matmul in moe_ops.h):
//
//     out[m,n] = sum_kb a_scale[m,kb] * b_scale[n/128,kb] * P_kb[m,n],   P_kb = the dot product over 128 of K
//
// The scales are arbitrary fp32 numbers, so the tensor cores cannot apply them (their block scales are powers of two):
// P_kb is formed in tensor memory by four tcgen05.mma kind::f8f6f4 (K = 32 each) and added up in registers, one fp32
// fused multiply-add a value and block of K. Two accumulator buffers in tensor memory (all of it with 256 columns a tile,
// half of it with 128) let the product of block kb + 1 run while eight warps take block kb out. A lane is a row of a and a
// warp's columns lie in one block of b, so a warp needs one factor a lane and block.
//
// Warp roles (384 threads): warp 0 TMA producer, warp 1 tensor-memory allocator and MMA issuer, warp 2 the groups' table,
// warps 4-11 take the products out (warp w the lanes 32 * (w % 4) .., warps 4-7 the first half of the tile's columns, 8-11
// the second). With 256 columns a tile these eight need 128 registers for their sums and 64 for the values on their way
// from tensor memory, so they take registers from the other four warps.
//
// Measured, 8192 x 4096 x 7168 to bf16: 188 us in short runs, 199 in a steady one at the power cap, 206 among other work (2.3-2.6
// PFLOP/s; 54 % of the tensor pipe). A buffer's way round (MMA, its commit, the warps' reads, their release) holds back the two
// buffers, for which tensor memory has room here: 840-860 cycles a block of K, reckoned from the steady run's time and clock; the same loop
// without the eight warps' work takes 144 us. Few rows (1 x 4096 x
// 7168: 11 us a call, 8.8 on the device, 29 MB) are bound by start-up, two buffers in turn and the cluster's sum around 14 blocks a
// CTA. Few rows of many groups are not split over K: 64 rows, 21 groups with rows, 4096 x 2048: 41 us for 177 MB (0.65 of the copy
// rate); 6 groups, 512 x 7168: 23 us for 22 MB (0.15), 24 CTAs that walk all of K alone.
//
// Every wait is bounded (2 s); on time-out the CTA records MOE_ERR_TIMEOUT and leaves its loops.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "group_tiles.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
// registers of warps 0-3 and 4-11: 128 * 40 + 256 * 232 = 384 * 168, what the launch holds
constexpr int kLaunchRegs = 168, kFewRegs = 40, kManyRegs = 232;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kMaxGroups = 1024;
constexpr int kPadRow = 17;  // floats of a staged row of 16 columns
constexpr int kTmemCols = 512;

struct Args {
    const float* a_scale;
    const float* b_scale;
    const int32_t* offsets;
    void* out;
    int32_t* hdr;
    int64_t out_stride;
    int M, N, groups, kb_count, nb_count;
    int n_tiles;
    int split;  // CTAs of a cluster that share a tile's blocks of K (one-CTA tiles only)
    bool vec;   // rows of out start on 32-byte boundaries
};

// kCtas 2: a pair of CTAs on one tile of 256 rows (cta_group::2), each holding 128 rows of a and half of the tile's rows of
// b. kARows: rows of a that are loaded (below 128 the accumulator's other rows hold sums nobody reads).
template <int kCtas_, int kBN_, int kARows_, int kStages_>
struct Cfg {
    static constexpr int kCtas = kCtas_, kBN = kBN_, kARows = kARows_, kStages = kStages_;
    static constexpr int kABytes = kARows * 128;
    static constexpr int kBRows = kBN / kCtas;
    static constexpr int kStageBytes = kABytes + kBRows * 128;
    static constexpr int kTileRows = 128 * kCtas;
    static constexpr int kCols = kBN / 2;  // columns of an epilogue warp
    static constexpr int kBarOff = kStages * kStageBytes;
    static constexpr int kNumBars = 2 * kStages + 2;
    static constexpr int kMiscOff = kBarOff + 8 * ((kNumBars + 1) & ~1);
    static constexpr int kTabOff = kMiscOff + 16;  // tile_off [groups + 1], lo [groups], hi [groups]
    static constexpr int kPadOff = kTabOff + 4 * (3 * kMaxGroups + 4);
    static constexpr size_t kSmem = 1024 + (size_t)kPadOff + 4 * kEpiWarps * 32 * kPadRow;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kCols % 32 == 0 && kCols <= 128, "tile");
    static_assert(kStageBytes >= 128 * 128, "the MMA reads 128 rows from the start of a stage");
    static_assert(kStages * kStageBytes >= 128 * kBN * 4 || kCtas == 2, "split sums use the stages' memory");
};

struct Tile {
    int g, n0, row0, hi;  // columns from n0 of group g; rows [row0, hi)
};

template <class C>
__device__ __forceinline__ Tile decode(int64_t t, const int* tab, int groups, int n_tiles) {
    const GroupTile f = find_group_tile(t, tab, groups, n_tiles, C::kTileRows);
    return {f.g, f.n_tile * C::kBN, f.row0, f.hi};
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, bool pair) {
    if (pair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// Arrives on a barrier of either CTA of the pair, ordered after this warp's reads of tensor memory (tcgen05.wait::ld and
// the fence before) and after nothing else: a release at cluster scope waits for the warp's loads and stores and took four
// fifths of the kernel's time.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// (x, y) += (p, q) * (s, s): one instruction for two values
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t p, uint32_t q, uint64_t s) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(p), "r"(q));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    return (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
}
template <typename Out>
__device__ __forceinline__ void store_out(void* base, int64_t i, float v) {
    if constexpr (sizeof(Out) == 2) static_cast<uint16_t*>(base)[i] = float_to_bf16_bits(v);
    else static_cast<float*>(base)[i] = v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Where column c of row r of a partial sum is kept: rows are turned by two columns each, so that the 32 rows of a warp
// write to different banks.
template <class C>
__device__ __forceinline__ int split_col(int r, int c) {
    return (c + 2 * r) & (C::kBN - 1);
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

template <class C, typename Out>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Args p) {
    constexpr bool kPair = C::kCtas == 2;
    constexpr int kStages = C::kStages;
    // kind::f8f6f4: fp32 sums (bit 4), e4m3 x e4m3, both K-major, N >> 3 (bits 17-22), M >> 4 (24-28)
    constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(C::kBN >> 3) << 17) | ((uint32_t)(C::kTileRows >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t bars = base + C::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto done_bar = [&](int s) { return bars + 8u * (kStages + s); };      // the stage's MMAs are finished
    auto free_bar = [&](int a) { return bars + 8u * (2 * kStages + a); };  // accumulator a has been read
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    int* tab = reinterpret_cast<int*>(smem + C::kTabOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = kPair ? 1 : p.split;
    const int share = kPair ? 2 : split;  // CTAs of a cluster
    const uint32_t rank = share > 1 ? cluster_ctarank() : 0u;
    const bool even = !kPair || rank == 0;
    const int64_t first = blockIdx.x / share, step = gridDim.x / share;
    const int kb0 = kPair ? 0 : (int)((int64_t)p.kb_count * rank / split);
    const int kb1 = kPair ? p.kb_count : (int)((int64_t)p.kb_count * (rank + 1) / split);

    if (warp == 2) write_group_tiles(p.offsets, p.M, p.groups, C::kTileRows, tab, lane);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(done_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) mbar_init(free_bar(a), kEpiWarps * C::kCtas);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
    }
    if (warp == 1) {
        if constexpr (kPair) tmem_alloc_pair(smem_u32(tmem_holder), kTmemCols);
        else tmem_alloc(smem_u32(tmem_holder), kTmemCols);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const int64_t total = (int64_t)tab[p.groups] * p.n_tiles;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0 && lane == 0) {
            int it = 0;
            bool ok = true;
            for (int64_t t = first; t < total && ok; t += step) {
                const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
                const int arow = tl.row0 + (kPair ? (int)rank * 128 : 0);
                const int brow = tl.g * p.N + tl.n0 + (kPair ? (int)rank * C::kBRows : 0);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(done_bar(s), ((uint32_t)(it / kStages) & 1u) ^ 1u, p.hdr, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * C::kStageBytes, sb = sa + C::kABytes;
                    if constexpr (kPair) {
                        const uint32_t fb = mapa_shared(full_bar(s), 0);
                        if (even) mbar_arrive_expect_tx(full_bar(s), 2 * C::kStageBytes);
                        tma_load_2d_pair(sa, &tmA, kb * 128, arow, fb);
                        tma_load_2d_pair(sb, &tmB, kb * 128, brow, fb);
                    } else {
                        mbar_arrive_expect_tx(full_bar(s), C::kStageBytes);
                        tma_load_2d(sa, &tmA, kb * 128, arow, full_bar(s));
                        tma_load_2d(sb, &tmB, kb * 128, brow, full_bar(s));
                    }
                }
            }
            // drain: every copy issued has landed (bounded)
            if (even)
                for (int j = it - kStages < 0 ? 0 : it - kStages; j < it; ++j)
                    if (!mbar_drain(full_bar(j % kStages), (uint32_t)(j / kStages) & 1u, p.hdr)) break;
        } else if (warp == 1 && even) {
            // the whole warp walks the loop and one elected lane issues: in a branch of a single lane the compiler cannot
            // tell that the operands are the same for the warp, and each MMA costs some 60 cycles to issue
            const uint64_t ad0 = kmajor_desc(base, 0), bd0 = kmajor_desc(base + C::kABytes, 0);
            int it = 0;
            bool ok = true;
            for (int64_t t = first; t < total && ok; t += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % kStages, a = it & 1;
                    ok = mbar_wait(full_bar(s), (uint32_t)(it / kStages) & 1u, p.hdr, abort_flag) &&
                         mbar_wait(free_bar(a), ((uint32_t)(it >> 1) & 1u) ^ 1u, p.hdr, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t off = (uint64_t)((s * C::kStageBytes) >> 4);
                        const uint32_t d = tmem_base + (uint32_t)(a * C::kBN);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma_f8(d, ad0 + off + 2 * kk, bd0 + off + 2 * kk, kIdesc, kk != 0, kPair);
                        // one commit a block, for the producer and the epilogue alike
                        if constexpr (kPair) tc2_commit_mc(done_bar(s), 0x3);
                        else tc_commit(done_bar(s));
                    }
                    __syncwarp();
                }
            }
            // drain: every MMA issued has completed before tensor memory is freed
            if (it > 0) mbar_drain(done_bar((it - 1) % kStages), (uint32_t)((it - 1) / kStages) & 1u, p.hdr);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int q = warp & 3, half = (warp - 4) >> 2;
        float* pad = reinterpret_cast<float*>(smem + C::kPadOff) + (warp - 4) * 32 * kPadRow;
        int it = 0;
        bool ok = true;
        for (int64_t t = first; t < total && ok; t += step) {
            const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
            const int wrow = tl.row0 + (kPair ? (int)rank * 128 : 0) + q * 32;  // the warp's first row
            const int row = wrow + lane, col0 = tl.n0 + half * C::kCols;
            const bool live = wrow < tl.hi && col0 < p.N;  // the warp has something to add up
            const float* sa = p.a_scale + (int64_t)min(row, tl.hi - 1) * p.kb_count;
            const float* sb = p.b_scale + ((int64_t)tl.g * p.nb_count + min(col0 / 128, p.nb_count - 1)) * p.kb_count;
            uint64_t acc[C::kCols / 2];
#pragma unroll
            for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
            float sa_next = kb0 < kb1 ? __ldg(sa + kb0) : 0.0f, sb_next = kb0 < kb1 ? __ldg(sb + kb0) : 0.0f;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int a = it & 1, s = it % kStages;
                const uint32_t factor = __float_as_uint(sa_next * sb_next);
                uint64_t s2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "r"(factor));
                const int next = min(kb + 1, kb1 - 1);  // on their way during this block
                sa_next = __ldg(sa + next);
                sb_next = __ldg(sb + next);
                ok = mbar_wait(done_bar(s), (uint32_t)(it / kStages) & 1u, p.hdr, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                auto release = [&]() {  // the buffer's values are in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kPair) mbar_arrive_pair(mapa_shared(free_bar(a), 0));
                        else mbar_arrive(free_bar(a));
                    }
                };
                if (live) {
                    const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * C::kBN + half * C::kCols);
                    // kChunk columns at a time, the next ones on their way while these are added
                    constexpr int kChunk = 16, kChunks = C::kCols / kChunk;
                    uint32_t r[2][kChunk];
                    tmem_ld16(ta, r[0]);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        tmem_ld_wait();
                        if (c + 1 < kChunks) tmem_ld16(ta + kChunk * (c + 1), r[(c + 1) & 1]);
                        else release();
#pragma unroll
                        for (int j = 0; j < kChunk / 2; ++j)
                            fma2(acc[c * (kChunk / 2) + j], r[c & 1][2 * j], r[c & 1][2 * j + 1], s2);
                    }
                } else {
                    release();
                }
            }
            if (!ok) break;
            if (split > 1) {
                // the partial sums go where the stages were (all of them have been read); [row][column]
                if (live) {
                    float* dst = reinterpret_cast<float*>(smem) + (q * 32 + lane) * C::kBN;
#pragma unroll
                    for (int j = 0; j < C::kCols / 2; ++j)
                        *reinterpret_cast<float2*>(dst + split_col<C>(q * 32 + lane, half * C::kCols + 2 * j)) = unpack2(acc[j]);
                }
            } else if (live) {
                const bool mine = row < tl.hi;
#pragma unroll
                for (int c = 0; c < C::kCols / 32; ++c) {
                    const int col = col0 + 32 * c;
                    if (p.vec && col + 32 <= p.N) {
                        Out* dst = static_cast<Out*>(p.out) + (int64_t)(mine ? row : wrow) * p.out_stride + col;
                        uint32_t w[32];
                        if constexpr (sizeof(Out) == 2) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 v = unpack2(acc[c * 16 + j]);
                                w[j] = bf16x2(v.x, v.y);
                            }
                            st_global_v8_if(mine, dst, w);
                            st_global_v8_if(mine, dst + 16, w + 8);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 v = unpack2(acc[c * 16 + j]);
                                w[2 * j] = __float_as_uint(v.x);
                                w[2 * j + 1] = __float_as_uint(v.y);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) st_global_v8_if(mine, dst + 8 * j, w + 8 * j);
                        }
                    } else {
                        // rows of any alignment: turned in shared memory so that half a warp writes 16 columns of one row
                        const int rows = min(32, tl.hi - wrow);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 v = unpack2(acc[c * 16 + 8 * h + j]);
                                pad[lane * kPadRow + 2 * j] = v.x;
                                pad[lane * kPadRow + 2 * j + 1] = v.y;
                            }
                            __syncwarp();
                            const int at = col + 16 * h + (lane & 15);
                            if (at < p.N)
                                for (int r = lane >> 4; r < rows; r += 2)
                                    store_out<Out>(p.out, (int64_t)(wrow + r) * p.out_stride + at, pad[r * kPadRow + (lane & 15)]);
                            __syncwarp();
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (share > 1) cluster_sync();  // pairs: neither leaves while the other uses its memory; splits: the sums are written
    tc_fence_after();
    if (!kPair && split > 1 && first < total) {
        // every CTA adds its share of the tile's values, over the cluster's CTAs in order
        const Tile tl = decode<C>(first, tab, p.groups, p.n_tiles);
        const int rows = min(128, tl.hi - tl.row0), cols = min(C::kBN, p.N - tl.n0);
        for (int i = (int)rank * kThreads + threadIdx.x; i < rows * C::kBN; i += split * kThreads) {
            const int r = i / C::kBN, c = i % C::kBN;
            if (c >= cols) continue;
            const uint32_t at = base + (uint32_t)(r * C::kBN + split_col<C>(r, c)) * 4u;
            float sum = 0.0f;
            for (int k = 0; k < split; ++k) sum += ld_cluster_f32(mapa_shared(at, (uint32_t)k));
            store_out<Out>(p.out, (int64_t)(tl.row0 + r) * p.out_stride + tl.n0 + c, sum);
        }
    }
    if (!kPair && split > 1) {
        __syncthreads();
        cluster_sync();  // nobody leaves while its sums are read
    }
    if (warp == 1) {
        if constexpr (kPair) tmem_dealloc_pair(tmem_base, kTmemCols);
        else tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------

using Large = Cfg<2, 256, 128, 5>;
using Wide = Cfg<1, 256, 128, 4>;
using Mid = Cfg<1, 128, 128, 5>;
using Few = Cfg<1, 128, 32, 8>;

template <class C, typename Out>
cudaError_t prepare_kernel(int* resident) {
    static int clusters[kMaxDevices];
    int device = 0;
    const cudaError_t err = once_per_device(&device, [](int dev) {
        cudaError_t e = cudaFuncSetAttribute(fp8_matmul_kernel<C, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e == cudaSuccess) e = check_register_split(reinterpret_cast<const void*>(fp8_matmul_kernel<C, Out>), kLaunchRegs);
        if (C::kCtas == 1 || e != cudaSuccess) return e;
        // pairs that can be resident at once (a pair needs two free SMs of one GPC)
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * std::max(1, tc_num_sms() / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&clusters[dev], fp8_matmul_kernel<C, Out>, &cfg) != cudaSuccess || clusters[dev] < 1) {
            (void)cudaGetLastError();
            clusters[dev] = std::max(1, tc_num_sms() / 2);
        }
        return e;
    });
    *resident = err == cudaSuccess ? clusters[device] : 0;
    return err;
}

template <class C, typename Out>
cudaError_t launch(const moe_fp8_matmul_args& a, Args p, int split, cudaStream_t s) {
    int resident = 0;
    cudaError_t err = prepare_kernel<C, Out>(&resident);
    if (err != cudaSuccess) return err;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {(uint64_t)a.K, (uint64_t)a.M}, db[2] = {(uint64_t)a.K, (uint64_t)a.N * a.groups};
    const uint64_t sa[1] = {(uint64_t)a.a_stride}, sb[1] = {(uint64_t)a.b_stride};
    const uint32_t boxa[2] = {128, (uint32_t)C::kARows}, boxb[2] = {128, (uint32_t)C::kBRows};
    if (!tc_make_map_nd(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.a, da, sa, boxa, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tc_make_map_nd(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.b, db, sb, boxb, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.n_tiles = (p.N + C::kBN - 1) / C::kBN;
    p.split = split;
    // row tiles: at most one unfilled per group (and none for groups without rows)
    const int64_t row_tiles = (a.M + C::kTileRows - 1) / C::kTileRows + std::min<int64_t>(a.groups - 1, a.M);
    const int64_t tiles = row_tiles * p.n_tiles;
    const int share = C::kCtas == 2 ? 2 : split;
    const int64_t clusters = split > 1 ? tiles : std::min<int64_t>(tiles, C::kCtas == 2 ? resident : tc_num_sms());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * share));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)share;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = share > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fp8_matmul_kernel<C, Out>, ma, mb, p);
}

template <typename Out>
cudaError_t launch_out(const moe_fp8_matmul_args& a, const Args& p, cudaStream_t s) {
    const int sms = tc_num_sms();
    // pairs: many rows a group and enough tiles of 256 x 256 (8192 x 4096 x 7168: 188 us, 197 with tiles of 128 x 256)
    if (a.M / a.groups >= 512 && ((a.M + 255) / 256) * ((a.N + 255) / 256) * 4 >= sms) return launch<Large, Out>(a, p, 1, s);
    // tiles of 128 x 256 fill shared memory with a quarter less than those of 128 x 128 and are taken where they give every SM one
    // (4099 rows of 32 groups, N 4096, K 2048: 59 us against 70; 1000 x 2112 x 7168, 72 tiles: 31 us against 23)
    const int64_t row_tiles = (a.M + 127) / 128 + (a.groups > 1 ? std::min<int64_t>(a.groups, a.M) / 2 : 0);
    if (row_tiles * ((a.N + 255) / 256) >= sms) return launch<Wide, Out>(a, p, 1, s);
    // few tiles: the blocks of K are shared by a cluster's CTAs as long as all tiles run at once
    int split = 1;
    const int64_t tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (a.groups == 1)
        while (split < 8 && tiles * split * 2 <= sms && p.kb_count >= split * 4) split *= 2;
    if (a.groups == 1 && a.M <= 32) return launch<Few, Out>(a, p, split, s);
    return launch<Mid, Out>(a, p, split, s);
}

}  // namespace

size_t fp8_matmul_workspace(int64_t, int64_t, int64_t, int) { return sizeof(int32_t) * kOpsHeaderInts; }

cudaError_t launch_fp8_matmul(const moe_fp8_matmul_args& a, void* workspace, cudaStream_t s) {
    if (a.M == 0) return cudaSuccess;
    Args p = {};
    p.a_scale = a.a_scale;
    p.b_scale = a.b_scale;
    p.offsets = a.offsets;
    p.out = a.out;
    p.hdr = static_cast<int32_t*>(workspace);
    p.out_stride = a.out_stride;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.groups = a.groups;
    p.kb_count = (int)((a.K + 127) / 128);
    p.nb_count = (int)((a.N + 127) / 128);
    const int64_t size = a.out_type == MOE_TYPE_BF16 ? 2 : 4;
    p.vec = !((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.out_stride * size)) & 31);
    return a.out_type == MOE_TYPE_BF16 ? launch_out<__nv_bfloat16>(a, p, s) : launch_out<float>(a, p, s);
}

}  // namespace moe
