// Product of int8 matrices with a scale for each row of either (moe_int8_matmul in moe_ops.h):
//
//     out[m,n] = (C[m,n] * b_scale[n]) * a_scale[m],   C = a . b^T exactly
//
// The chip has no integer kind of tcgen05.mma, and mma.sync on int8 and dp4a both run at 150 TOP/s, a sixteenth of the f16 rate. So the
// codes are multiplied as f16 numbers, which hold them exactly: a product is below 2^14 in magnitude and an fp32 sum of 1024 of
// them at most 2^24, still an exact integer. At least every 1024 of K the sums are taken out of tensor memory and added up as
// integers in registers, which makes C exact for every input.
//
// Codes become f16 inside the kernel, on their way from shared memory: the operands are read from HBM as bytes, and neither a pass of its
// own nor twice the traffic is needed. Of the two operands the weights (rows of b, the M side of the MMA) go to tensor
// memory, which the MMA takes its first operand from, and the tokens (rows of a, the N side) back to shared memory: what
// bounds such a kernel is shared memory's 128 bytes a cycle (bytes in by TMA, out to the converters, f16 tokens in, and out to the
// MMA), and weights that went back too would add half as much again.
//
// Warp roles: warp 0 TMA producer, warp 1 tensor-memory allocator and MMA issuer, warp 2 the groups' table, warp 3 a split tile's scales,
// warps 4-11 take sums out and write results, the others (8 or 16) convert.
//
// Measured, 8192 x 4096 x 7168 to bf16: 288 us (1.67 PFLOP/s; 0.86 of cuBLAS's bf16 burst rate, 0.94 of its sustained one). A stage of 128 of
// K is 1024 cycles of MMAs on a 256 x 256 pair tile and takes some 1350: the same 1024 cycles of shared memory (32 KB each way in,
// out, in and out) and half of the schedulers' slots contend with them; without converters and epilogue the loop takes 220 us. 4099
// rows of 32 groups, 4096 x 2048: 91 us, 2.6 TB/s of weights (28 groups have rows); a stage is 512 cycles of MMAs on a 256 x 128 tile and takes 1100
// (ALU 61 % busy, tensor pipe 32 %). 133 x 2112 x 7168: 17 us, 14 stages a CTA at 980 cycles, 3 us before the first operands, 3 for the
// cluster's sum.
// What it took, on the first of these: 436 us with a forwarder that released everything of the odd CTA's at cluster scope (850 cycles a stage);
// 404 with converters of both CTAs arriving themselves; 310 with sums taken out in pauses of two steps and converters of both operands
// in every warp; 305 with one commit a stage; 292 without a conversion to integers of every value of every chunk. Slower: sums read by
// warps that sleep between their looks (315), packed bf16 stores of two rows (305), spinning tests instead of waits (298).
//
// Every wait is bounded (2 s); on time-out the CTA records MOE_ERR_TIMEOUT and leaves its loops.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "group_tiles.cuh"
#include "int8_matmul.h"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kEpiWarps = 8;
constexpr int kFewRegs = 48, kConvRegs = 56;  // registers of warps 0-3 and of the converters
constexpr int kTmemCols = 512;
constexpr int kMaxSplit = 8;  // CTAs of a cluster that share a tile
constexpr int kStageK = 128;                  // codes of K in a stage
constexpr int kChunkStages = 1024 / kStageK;  // stages of an exact fp32 sum

struct Args {
    const float* a_scale;
    const float* b_scale;
    const int32_t* offsets;
    void* out;
    int32_t* hdr;
    int64_t out_stride;
    int M, N, groups, kb_count;
    int n_tiles;
    int split;  // CTAs of a cluster that share a tile's stages (one-CTA tiles without groups only)
};

// A tile is 128 * kCtas weight rows by kHalves * kN tokens. kCtas 2: a pair of CTAs (cta_group::2), each holding 128 of the weight rows
// and half of the tokens of every MMA. kHalves 2: two MMAs of kN tokens a step, each with a sum of its own; 1: one, whose
// sum changes between two buffers from chunk to chunk. kRaw, kOps: stages of bytes, and of operands. kConvWarps: converters; kEpiRegs,
// kLaunchRegs: registers of a thread of the warps that hold the sums, and of every thread at launch.
template <int kCtas_, int kN_, int kHalves_, int kRaw_, int kOps_, int kConvWarps_, int kEpiRegs_, int kLaunchRegs_>
struct Cfg {
    static constexpr int kConvWarps = kConvWarps_, kEpiRegs = kEpiRegs_, kLaunchRegs = kLaunchRegs_;
    static constexpr int kThreads = 32 * (4 + kEpiWarps + kConvWarps);
    static constexpr int kGroups = kConvWarps / 4;  // of converters, half a stage each in turn
    static_assert(128 * kFewRegs + 32 * kEpiWarps * kEpiRegs + 32 * kConvWarps * kConvRegs <= kThreads * kLaunchRegs, "register split");
    static_assert(kThreads * kLaunchRegs <= 65536 && (kGroups == 2 || kGroups == 4), "warps");
    static constexpr int kCtas = kCtas_, kN = kN_, kHalves = kHalves_, kRaw = kRaw_, kOps = kOps_;
    static constexpr int kStep = kHalves;                   // stages of a step
    static constexpr int kTokens = kN * kHalves;
    static constexpr int kBRows = kTokens / kCtas, kHalfRows = kN / kCtas;
    static constexpr int kRawA = 128 * kStageK, kRawBytes = kRawA + kBRows * kStageK;
    static constexpr int kAtomBytes = kBRows * 128, kOpBytes = 2 * kAtomBytes;  // tokens in f16: two swizzled atoms of 64 of K
    static constexpr int kOpOff = kRaw * kRawBytes;
    static constexpr int kBarOff = kOpOff + kOps * kOpBytes;
    static constexpr int kNumBars = 2 * kRaw + 2 * kOps + 5;
    static constexpr int kMiscOff = kBarOff + 8 * ((kNumBars + 1) & ~1);
    static constexpr int kTabOff = kMiscOff + 16;
    static constexpr int kMaxTab = 232448 - 1024 - kTabOff;
    static constexpr int kScales = kCtas == 1 ? 128 + kTokens : 0;  // floats of a split tile's scales, behind the table
    static size_t smem(int groups) { return 1024 + (size_t)kTabOff + 4 * (3 * groups + 4) + 4 * kScales; }
    static constexpr int kCols = kHalves == 2 ? kN : kN / 2;  // sums of a lane of the epilogue
    static constexpr int kTmemA = 2 * kN;                     // first column of the weights' stages, kStageK / 2 columns each
    static constexpr int kMaxGroups = (kMaxTab - 4 * kScales) / 12 - 2;  // whose table fits
    static constexpr int kMine = kBRows / 32;                 // 16-byte chunks of a token row that a converter thread takes
    static_assert(kMaxGroups >= 1, "shared memory");
    static_assert(kTmemA + kOps * (kStageK / 2) <= kTmemCols, "tensor memory");
    static_assert(kCols % 16 == 0 && kCols <= 128 && kMine >= 1 && kMine <= 4 && kBRows == 32 * kMine, "tile");
    static_assert(kOps >= 2 * kStep, "two steps of operands");
    // A slot of bytes is waited for by the same groups in every round: bytes may land out of order, and a group that waits for the round after one
    // it has not seen land would pass for the wrong parity. (Slots of operands are freed in order, so their waits may change hands.)
    static_assert(kRaw % (kGroups / 2) == 0 && kOps >= kGroups / 2, "rounds of the slots");
    static_assert(kCtas == 2 || kBarOff >= 4 * 128 * kTokens, "split sums use the stages' memory");
};

struct Tile {
    int g, n0, row0, hi;  // weight rows from n0 of group g; tokens [row0, hi)
    int n;                // tokens of an MMA
};

template <class C>
__device__ __forceinline__ Tile decode(int64_t t, const int* tab, int groups, int n_tiles) {
    const GroupTile f = find_group_tile(t, tab, groups, n_tiles, C::kTokens);
    // (the N of an MMA is a multiple of 16)
    return {f.g, f.n_tile * 128 * C::kCtas, f.row0, f.hi, C::kHalves == 2 ? C::kN : min(C::kN, (f.hi - f.row0 + 15) & ~15)};
}

// Whether the sum of a half is taken out after step d of n. The halves' MMAs alternate as 0 1 | 1 0 | 0 1 | ..., so the half that was first
// in step 0 has a gap of two steps of the other half's after every even step, the other one after every odd step: the sums are
// taken out in these gaps. At most kSteps steps, 1024 of K, are added up.
template <class C>
__device__ __forceinline__ bool taken_out(bool first, int d, int n) {
    constexpr int kSteps = kChunkStages / C::kStep;
    return d == n - 1 || d % kSteps == kSteps - (first ? 2 : 1);
}

// four codes as f16 numbers: c + 128 is put into the fraction of 1024, from which 1152 is subtracted
__device__ __forceinline__ void to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// 16 consecutive 32-bit columns of this thread's lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// D += A (128 or 256 rows, tensor memory) x B (shared memory), K = 16
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, bool pair) {
    if (pair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

// A test and a bounded wait that begins with it: a try_wait costs 170-280 cycles when the phase has long completed, a test a fraction.
// kCluster: for a barrier that the other CTA of the pair, or its MMAs' commits, arrive on, too (what that CTA did is seen).
template <bool kCluster = false>
__device__ __forceinline__ bool completed(uint32_t bar, uint32_t parity) {
    if constexpr (!kCluster) return mbar_test(bar, parity);
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int32_t* hdr, volatile int* abort_flag) {
    if (completed<kCluster>(bar, parity)) return true;
    if (!mbar_wait(bar, parity, hdr, abort_flag)) return false;
    return !kCluster || completed<kCluster>(bar, parity);
}

// Arrives on a barrier of either CTA of the pair for operands that this warp has written to its own CTA's shared memory (each lane's made visible
// to the MMA by its fence.proxy.async) and tensor memory (tcgen05.wait::st and the fence after it, which an execution order of
// cluster scope completes). The fence releases the former to the pair: it covers shared memory alone, so it waits for no access to
// any other. A release of cluster scope of everything (arrive.release or fence.acq_rel) took 463 and 469 us where this takes 288
// (8192 x 4096 x 7168), 132 and 135 where this takes 91 (4099 rows of 32 groups).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
        : "memory");
}

// Arrives on a barrier of either CTA of the pair after this warp's reads of tensor memory alone: tcgen05.wait::ld and the fence after it order
// them, with the fence that the MMA warp has after its wait.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <typename Out>
__device__ __forceinline__ void store_if(bool on, Out* p, float v) {
    if constexpr (sizeof(Out) == 2) st_global_u16_if(on, p, float_to_bf16_bits(v));
    else asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.f32 [%1], %2;\n\t}" ::"r"((int)on), "l"(p), "f"(v));
}

template <class C, typename Out>
__global__ void __launch_bounds__(C::kThreads, 1)
    int8_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Args p) {
    constexpr bool kPair = C::kCtas == 2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t bars = base + C::kBarOff;
    auto raw_full = [&](int s) { return bars + 8u * s; };                                 // bytes have landed
    auto raw_free = [&](int s) { return bars + 8u * (C::kRaw + s); };                     // and have been read
    auto op_full = [&](int s) { return bars + 8u * (2 * C::kRaw + s); };                  // operands are written
    auto op_free = [&](int s) { return bars + 8u * (2 * C::kRaw + C::kOps + s); };        // and their MMAs finished
    auto acc_full = [&](int a) { return bars + 8u * (2 * C::kRaw + 2 * C::kOps + a); };   // a sum is ready
    auto acc_free = [&](int a) { return bars + 8u * (2 * C::kRaw + 2 * C::kOps + 2 + a); };  // and has been read
    const uint32_t end_bar = bars + 8u * (C::kNumBars - 1);                                  // every MMA is finished
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    int* tab = reinterpret_cast<int*>(smem + C::kTabOff);
    float* tile_scales = reinterpret_cast<float*>(tab + 3 * p.groups + 4);  // (split tiles) of 128 weight rows, then of the tokens

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = kPair ? 1 : p.split;
    const int share = kPair ? 2 : split;  // CTAs of a cluster
    const uint32_t rank = share > 1 ? cluster_ctarank() : 0u;
    const int half_cta = kPair ? (int)rank : 0;
    const bool even = half_cta == 0;
    const int64_t first = blockIdx.x / share, step = gridDim.x / share;
    const int kb0 = kPair ? 0 : (int)((int64_t)p.kb_count * rank / split);
    const int kb1 = kPair ? p.kb_count : (int)((int64_t)p.kb_count * (rank + 1) / split);
    const int steps = (kb1 - kb0 + C::kStep - 1) / C::kStep;

    // bytes of stage kb of the tile whose weight rows begin at wrow and tokens at trow, into slot s
    auto load_stage = [&](int s, int kb, int wrow, int trow) {
        const uint32_t dst = base + s * C::kRawBytes;
        mbar_arrive_expect_tx(raw_full(s), C::kRawBytes);
        tma_load_2d(dst, &tmB, kb * kStageK, wrow, raw_full(s));
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
            tma_load_2d(dst + C::kRawA + h * C::kHalfRows * kStageK, &tmA, kb * kStageK, trow + h * C::kN, raw_full(s));
    };
    int early = 0;  // stages that the producer has sent for already

    if (warp == 2) write_group_tiles(p.offsets, p.M, p.groups, C::kTokens, tab, lane);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kRaw; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_free(s), 8);  // (two groups of converters)
        }
        for (int s = 0; s < C::kOps; ++s) {
            mbar_init(op_full(s), 8 * C::kCtas);  // (the even CTA's; the odd one's is not used)
            mbar_init(op_free(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_free(a), kEpiWarps / C::kHalves * C::kCtas);
        }
        mbar_init(end_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // without groups the first tile is known before the table: its first stages are on their way while the rest is set up (in this CTA's
        // memory, on barriers that this thread has just made)
        if (!p.offsets && first < (int64_t)((p.M - 1) / C::kTokens + 1) * p.n_tiles) {
            const int mt = (p.M - 1) / C::kTokens + 1, row0 = (int)(first % mt) * C::kTokens;
            const int n = C::kHalves == 2 ? C::kN : min(C::kN, (p.M - row0 + 15) & ~15);
            for (early = 0; early < min(C::kRaw, kb1 - kb0); ++early)
                load_stage(early, kb0 + early, (int)(first / mt) * 128 * C::kCtas + half_cta * 128, row0 + half_cta * (n / C::kCtas));
        }
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
            int it = 0, s = 0;
            uint32_t parity = 1;
            bool ok = true;
            for (int64_t t = first; t < total && ok; t += step) {
                const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
                const int wrow = tl.g * p.N + tl.n0 + half_cta * 128;
                const int trow = tl.row0 + half_cta * (tl.n / C::kCtas);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    if (it >= early) {
                        if (!wait_for(raw_free(s), parity, p.hdr, abort_flag)) {
                            ok = false;
                            break;
                        }
                        load_stage(s, kb, wrow, trow);
                    }
                    if (++s == C::kRaw) s = 0, parity ^= 1u;
                }
            }
            // drain: every copy issued has landed (bounded)
            for (int j = it - C::kRaw < 0 ? 0 : it - C::kRaw; j < it; ++j)
                if (!mbar_drain(raw_full(j % C::kRaw), (uint32_t)(j / C::kRaw) & 1u, p.hdr)) break;
        } else if (warp == 1 && even) {
            // the whole warp walks the loop and one elected lane issues
            const uint64_t bd0 = kmajor_desc(base + C::kOpOff, 0);
            int it = 0, sums[2] = {0, 0};
            bool ok = true;
            bool ready_op = false;  // operand stage `it` was seen written, by a test a turn ahead
            auto wait_ops = [&](int i) {
                if (!__all_sync(0xffffffffu, ready_op))
                    ok = __all_sync(0xffffffffu, wait_for<kPair>(op_full(i % C::kOps), (uint32_t)(i / C::kOps) & 1u, p.hdr, abort_flag));
                if (ok) tc_fence_after();
                return ok;
            };
            auto test_ops = [&](int i) { ready_op = completed<kPair>(op_full(i % C::kOps), (uint32_t)(i / C::kOps) & 1u); };
            auto wait_acc = [&](int a, int times) {
                ok = __all_sync(0xffffffffu, wait_for<kPair>(acc_free(a), ((uint32_t)times & 1u) ^ 1u, p.hdr, abort_flag));
                if (ok) tc_fence_after();
                return ok;
            };
            // the MMAs of operand stage i and half h into buffer a; then what is finished with them
            auto issue = [&](int i, int h, int a, uint32_t idesc, bool fresh, bool frees, bool ready) {
                const int s = i % C::kOps;
                if (elect_one()) {
                    const uint32_t d = tmem_base + (uint32_t)(a * C::kN), wa = tmem_base + (uint32_t)(C::kTmemA + s * (kStageK / 2));
                    const uint64_t bd = bd0 + (uint64_t)((s * C::kOpBytes + h * C::kHalfRows * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kStageK / 16; ++kk)
                        mma_ta(d, wa + 8 * kk, bd + (uint64_t)((kk / 4 * C::kAtomBytes + kk % 4 * 32) >> 4), idesc, !(fresh && kk == 0), kPair);
                    if constexpr (kPair) {
                        if (frees) tc2_commit_mc(op_free(s), 0x3);
                        if (ready) tc2_commit_mc(acc_full(a), 0x3);
                    } else {
                        if (frees) tc_commit(op_free(s));
                        if (ready) tc_commit(acc_full(a));
                    }
                }
                __syncwarp();
            };
            int lead = 0;  // the half whose MMAs come first in the tile
            for (int64_t t = first; t < total && ok; t += step) {
                const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
                // kind::f16: fp32 sums (bit 4), f16 x f16, both K-major, N >> 3 (bits 17-22), M >> 4 (24-28)
                const uint32_t idesc = (1u << 4) | ((uint32_t)(tl.n >> 3) << 17) | ((uint32_t)(8 * C::kCtas) << 24);
                if constexpr (C::kHalves == 1) {
                    for (int d = 0; d < steps && ok; ++d, ++it) {
                        const bool fresh = d % kChunkStages == 0, ready = d % kChunkStages == kChunkStages - 1 || d == steps - 1;
                        const int a = sums[0] & 1;
                        if (fresh && !wait_acc(a, sums[0] >> 1)) break;
                        if (!wait_ops(it)) break;
                        test_ops(it + 1);
                        issue(it, 0, a, idesc, fresh, true, ready);
                        if (ready) ++sums[0];
                    }
                } else {
                    uint32_t fresh = 3;  // bit h: the next MMA of half h begins a sum
                    for (int d = 0; d < steps && ok; ++d) {
                        const int n = min(C::kStep, kb1 - kb0 - d * C::kStep);
                        for (int o = 0; o < 2 && ok; ++o) {
                            const int h = lead ^ (d & 1) ^ o;
                            const bool out = taken_out<C>(h == lead, d, steps);
                            if ((fresh >> h & 1) && !wait_acc(h, sums[h])) break;
                            for (int i = 0; i < n; ++i) {
                                if (o == 0 && !wait_ops(it + i)) break;
                                if (o == 0 || i == n - 1) test_ops(o == 0 ? it + i + 1 : it + n);
                                issue(it + i, h, h, idesc, (fresh >> h & 1) && i == 0, o == 1, out && i == n - 1);
                            }
                            fresh = out ? fresh | 1u << h : fresh & ~(1u << h);
                            if (out) ++sums[h];
                        }
                        it += n;
                    }
                    lead ^= (steps - 1) & 1;  // the half that was first in the last step has had the longer pause
                }
            }
            // drain: every MMA issued has completed before shared and tensor memory are given up, after a time-out too
            if (elect_one()) {
                if constexpr (kPair) tc2_commit_mc(end_bar, 0x1);
                else tc_commit(end_bar);
            }
            __syncwarp();
            mbar_drain(end_bar, 0, p.hdr);
        } else if (warp == 3 && !kPair && split > 1 && first < total) {
            const Tile tl = decode<C>(first, tab, p.groups, p.n_tiles);
            for (int i = lane; i < 128; i += 32) tile_scales[i] = tl.n0 + i < p.N ? __ldg(p.b_scale + (int64_t)tl.g * p.N + tl.n0 + i) : 0.0f;
            for (int i = lane; i < C::kTokens; i += 32) tile_scales[128 + i] = tl.row0 + i < tl.hi ? __ldg(p.a_scale + tl.row0 + i) : 0.0f;
        }
    } else if (warp >= 4 + kEpiWarps) {  // (the last warps)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        // groups of four warps convert half a stage each, in turn: the chain of waits, loads, stores and fences is longer than the half's MMAs.
        // A warp has 32 weight rows (a row a lane: tensor memory gives a warp the 32 lanes of its place in four) and a fourth of
        // the tokens' chunks.
        const int q = warp & 3, group = (warp - 4 - kEpiWarps) >> 2, i = group & 1, id = q * 32 + lane;
        const int row = id % C::kBRows, chunk = id / C::kBRows * C::kMine;
        const uint32_t wsw = (uint32_t)(id & 7), sw = (uint32_t)(row & 7);
        const uint32_t tmem_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)C::kTmemA;
        int s = group >> 1;                  // stage of bytes, and its round
        uint32_t parity = 0;
        uint32_t turn = (uint32_t)s;         // of the operand stages
        int others = s;                      // stages of bytes until this group's next
        bool ok = true, landed = false, freed = true;  // tests made a turn ahead
        for (int64_t t = first; t < total && ok; t += step) {
            const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
            const bool mine = row < (C::kHalves == 2 ? C::kBRows : tl.n / C::kCtas);  // a token row that an MMA reads
            for (int kb = kb0; kb < kb1; ++kb) {
                if (others > 0) {
                    --others;
                    continue;
                }
                others = C::kGroups / 2 - 1;
                const uint32_t o = turn % C::kOps;
                if (!__all_sync(0xffffffffu, landed && freed)) {
                    ok = wait_for(raw_full(s), parity, p.hdr, abort_flag) &&
                         wait_for<kPair>(op_free(o), (turn / C::kOps & 1u) ^ 1u, p.hdr, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                tc_fence_after();
                const uint32_t wsrc = base + s * C::kRawBytes + id * kStageK, src = base + s * C::kRawBytes + C::kRawA + row * kStageK;
                // chunks of 16 bytes: 16 of K each
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = ld_shared16(wsrc + (((uint32_t)(4 * i + j) ^ wsw) << 4));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        to_f16(w[2 * h + j].x, f[8 * j + 0], f[8 * j + 1]);
                        to_f16(w[2 * h + j].y, f[8 * j + 2], f[8 * j + 3]);
                        to_f16(w[2 * h + j].z, f[8 * j + 4], f[8 * j + 5]);
                        to_f16(w[2 * h + j].w, f[8 * j + 6], f[8 * j + 7]);
                    }
                    tmem_st16(tmem_row + (uint32_t)(o * (kStageK / 2) + 32 * i + 16 * h), f);
                }
#pragma unroll
                for (int j = 0; j < C::kMine; ++j)
                    if (mine) w[j] = ld_shared16(src + (((uint32_t)(4 * i + chunk + j) ^ sw) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(raw_free(s));
                s += C::kGroups / 2;
                if (s >= C::kRaw) s -= C::kRaw, parity ^= 1u;
                turn += C::kGroups / 2;
                landed = completed(raw_full(s), parity);
                freed = completed<kPair>(op_free(turn % C::kOps), (turn / C::kOps & 1u) ^ 1u);
                const uint32_t dst = base + C::kOpOff + o * C::kOpBytes + i * C::kAtomBytes + row * 128;
#pragma unroll
                for (int j = 0; j < C::kMine; ++j) {
                    uint32_t u[8];
                    to_f16(w[j].x, u[0], u[1]);
                    to_f16(w[j].y, u[2], u[3]);
                    to_f16(w[j].z, u[4], u[5]);
                    to_f16(w[j].w, u[6], u[7]);
                    const uint32_t slot = (uint32_t)(2 * (chunk + j));  // 8 of K
                    if (mine) {
                        st_shared16(dst + ((slot ^ sw) << 4), u);
                        st_shared16(dst + (((slot + 1) ^ sw) << 4), u + 4);
                    }
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (kPair) mbar_arrive_remote(mapa_shared(op_full(o), 0));
                    else mbar_arrive(op_full(o));
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
        const int q = warp & 3, half = (warp - 4) >> 2;
        int sums = 0, lead = 0;
        bool ok = true;
        for (int64_t t = first; t < total && ok; t += step) {
            const Tile tl = decode<C>(t, tab, p.groups, p.n_tiles);
            const int n = tl.n0 + half_cta * 128 + q * 32 + lane;                            // the lane's weight row
            const int m0 = tl.row0 + half * C::kCols;                                        // its first token
            const int cols = C::kHalves == 2 ? C::kCols : min(C::kCols, tl.n - half * C::kCols);  // (multiples of 16; or none)
            const bool live = n - lane < p.N && m0 < tl.hi && cols > 0;
            // The sums so far, in fp32 as long as they are integers below 2^24 for certain (`room` is what a lane's next chunks may add up
            // to), as most sums are to the end; from then on (`wide`, a whole warp's) as integers: the conversion of every value of
            // every chunk runs at a sixteenth of the rate of an addition and held the MMAs up.
            uint32_t acc[C::kCols];
            bool wide = false;
            float room = 16777216.0f;
#pragma unroll
            for (int j = 0; j < C::kCols; ++j) acc[j] = 0;
            auto take = [&](int a, uint32_t parity) {
                ok = __all_sync(0xffffffffu, wait_for<kPair>(acc_full(a), parity, p.hdr, abort_flag));
                if (!ok) return;
                tc_fence_after();
                if (live) {
                    const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * C::kN + (C::kHalves == 2 ? 0 : half * C::kCols));
                    int from = 0;  // first group of 16 columns that is added as integers
                    if (!wide) {
                        from = C::kCols / 16;
                        float most = 0.0f;
#pragma unroll
                        for (int c = 0; c < C::kCols / 16; ++c) {
                            if (16 * c >= cols) break;
                            uint32_t r[16];
                            tmem_ld16(ta + 16 * c, r);
                            tmem_ld_wait();
                            float top = 0.0f;
#pragma unroll
                            for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(__uint_as_float(r[j])));
                            if (__any_sync(0xffffffffu, top > room)) {
                                from = c;
                                break;
                            }
                            most = fmaxf(most, top);
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[16 * c + j] = __float_as_uint(__uint_as_float(acc[16 * c + j]) + __uint_as_float(r[j]));
                        }
                        room -= most;
                        if (from < C::kCols / 16 && 16 * from < cols) {
                            wide = true;
#pragma unroll
                            for (int j = 0; j < C::kCols; ++j) acc[j] = (uint32_t)__float2int_rn(__uint_as_float(acc[j]));
                        }
                    }
                    if (wide) {
#pragma unroll
                        for (int c = 0; c < C::kCols / 16; ++c) {
                            if (16 * c >= cols) break;
                            if (c < from) continue;
                            uint32_t r[16];
                            tmem_ld16(ta + 16 * c, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[16 * c + j] += (uint32_t)__float2int_rn(__uint_as_float(r[j]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (kPair) mbar_arrive_relaxed(mapa_shared(acc_free(a), 0));
                    else mbar_arrive(acc_free(a));
                }
            };
            if constexpr (C::kHalves == 1) {
                for (int kb = kb0; kb < kb1 && ok; kb += kChunkStages, ++sums) take(sums & 1, (uint32_t)(sums >> 1) & 1u);
            } else {
                for (int d = 0; d < steps && ok; ++d)
                    if (taken_out<C>(half == lead, d, steps)) {
                        take(half, (uint32_t)sums & 1u);
                        ++sums;
                    }
                lead ^= (steps - 1) & 1;
            }
            if (!ok) break;
            if (split > 1) {
                // the partial sums go where the stages were (all of them have been read): [token][weight row]
                if (live) {
                    int* dst = reinterpret_cast<int*>(smem) + half * C::kCols * 128 + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < C::kCols; ++j) dst[j * 128] = wide ? (int)acc[j] : __float2int_rn(__uint_as_float(acc[j]));
                }
            } else if (live) {
                if (wide)
#pragma unroll
                    for (int j = 0; j < C::kCols; ++j) acc[j] = __float_as_uint((float)(int)acc[j]);
                const float bs = n < p.N ? __ldg(p.b_scale + (int64_t)tl.g * p.N + n) : 0.0f;
                const int rows = n < p.N ? min(tl.hi - m0, cols) : 0;
                Out* dst = static_cast<Out*>(p.out) + (int64_t)m0 * p.out_stride + n;
#pragma unroll
                for (int c = 0; c < C::kCols; c += 32) {
                    const float as = __ldg(p.a_scale + min(m0 + c + lane, tl.hi - 1));
#pragma unroll
                    for (int j = 0; j < 32; ++j, dst += p.out_stride)
                        store_if(c + j < rows, dst, int8_scaled(__uint_as_float(acc[c + j]), bs, __shfl_sync(0xffffffffu, as, j)));
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (share > 1) cluster_sync();  // pairs: neither leaves while the other uses its memory; splits: the sums are written
    tc_fence_after();
    if (!kPair && split > 1) {
        if (first < total) {
            // every CTA adds up its share of the tile's values, of four weight rows of a token at a time
            const Tile tl = decode<C>(first, tab, p.groups, p.n_tiles);
            const int rows = min(C::kTokens, tl.hi - tl.row0);
            for (int i = (int)rank * C::kThreads + threadIdx.x; i < rows * 32; i += split * C::kThreads) {
                const int j = i / 32, w = i % 32 * 4;  // token, and the first of the weight rows
                int v[kMaxSplit][4];
#pragma unroll
                for (int k = 0; k < kMaxSplit; ++k) {  // (all on their way at once)
                    if (k < split)
                        asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[k][0]), "=r"(v[k][1]), "=r"(v[k][2]), "=r"(v[k][3])
                                     : "r"(mapa_shared(base + (uint32_t)i * 16u, (uint32_t)k))
                                     : "memory");
                    else v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0;
                }
                Out* dst = static_cast<Out*>(p.out) + (int64_t)(tl.row0 + j) * p.out_stride + tl.n0 + w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int sum = 0;
#pragma unroll
                    for (int k = 0; k < kMaxSplit; ++k) sum += v[k][e];
                    store_if(tl.n0 + w + e < p.N, dst + e, int8_scaled((float)sum, tile_scales[w + e], tile_scales[128 + j]));
                }
            }
        }
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

using Large = Cfg<2, 128, 2, 3, 4, 8, 160, 96>;
using Pair = Cfg<2, 128, 1, 6, 4, 16, 104, 72>;
using Mid = Cfg<1, 128, 1, 3, 3, 8, 160, 96>;
using Small = Cfg<1, 64, 1, 6, 4, 16, 104, 72>;
static_assert(Pair::kMaxGroups >= 1024 && Mid::kMaxGroups >= 1024 && Small::kMaxGroups >= 1024, "tables of as many groups as a call takes");

// Attributes of the kernel on the current device; resident[s]: clusters of s CTAs that run at once there (of 2 for pairs; of each size that a
// tile may be split over, for the others). A cluster's CTAs share a GPC, so fewer fit than the SMs would hold.
template <class C, typename Out>
cudaError_t prepare_kernel(const int** resident) {
    static int clusters[kMaxDevices][kMaxSplit + 1];
    int device = 0;
    const cudaError_t err = once_per_device(&device, [](int dev) {
        cudaError_t e = cudaFuncSetAttribute(int8_matmul_kernel<C, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e == cudaSuccess) e = check_register_split(reinterpret_cast<const void*>(int8_matmul_kernel<C, Out>), C::kLaunchRegs);
        for (int size = C::kCtas; size <= (C::kCtas == 2 ? 2 : kMaxSplit) && e == cudaSuccess; ++size) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(size * std::max(1, tc_num_sms() / size));
            cfg.blockDim = dim3(C::kThreads);
            cfg.dynamicSmemBytes = C::smem(1);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = size;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&clusters[dev][size], int8_matmul_kernel<C, Out>, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                clusters[dev][size] = 0;
            }
        }
        if (clusters[dev][C::kCtas] < 1) clusters[dev][C::kCtas] = std::max(1, tc_num_sms() / C::kCtas);
        return e;
    });
    *resident = clusters[device];
    return err;
}

template <class C, typename Out>
cudaError_t launch(const moe_int8_matmul_args& a, Args p, cudaStream_t s) {
    const int* resident;
    const cudaError_t err = prepare_kernel<C, Out>(&resident);
    if (err != cudaSuccess) return err;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {(uint64_t)a.K, (uint64_t)a.M}, db[2] = {(uint64_t)a.K, (uint64_t)a.N * a.groups};
    const uint64_t sa[1] = {(uint64_t)a.a_stride}, sb[1] = {(uint64_t)a.b_stride};
    const uint32_t boxa[2] = {kStageK, (uint32_t)(C::kHalves == 2 ? C::kHalfRows : C::kBRows)}, boxb[2] = {kStageK, 128};
    if (!tc_make_map_nd(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.a, da, sa, boxa, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tc_make_map_nd(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.b, db, sb, boxb, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.n_tiles = (p.N + 128 * C::kCtas - 1) / (128 * C::kCtas);
    // row tiles: at most one unfilled per group (and none for groups without rows)
    const int64_t row_tiles = (a.M + C::kTokens - 1) / C::kTokens + std::min<int64_t>(a.groups - 1, a.M);
    const int64_t tiles = row_tiles * p.n_tiles;
    // few tiles: the stages are shared by as many CTAs of a cluster as all tiles' clusters run at once with, four stages each or more
    int split = 1;
    if (C::kCtas == 1 && a.groups == 1)
        for (int size = 2; size <= kMaxSplit && p.kb_count >= 4 * size; ++size)
            if (tiles <= resident[size]) split = size;
    p.split = split;
    const int share = C::kCtas == 2 ? 2 : split;
    const int64_t clusters = split > 1 ? tiles : std::min<int64_t>(tiles, resident[C::kCtas]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * share));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::smem(p.groups);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)share;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = share > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, int8_matmul_kernel<C, Out>, ma, mb, p);
}

// Tiles by sizes alone (times with N 4096, K 7168 where no other is given; `sms` 152 here)
template <typename Out>
cudaError_t launch_out(const moe_int8_matmul_args& a, const Args& p, cudaStream_t s) {
    const int sms = tc_num_sms();
    const int64_t n_tiles = (a.N + 255) / 256, rows = a.M / a.groups;
    // Few rows: 16 rows 13.0 us there and 14.5 on Small, 32 rows 22 and 14. Of groups, where Small has a CTA for less than every SM, but rows may all be
    // one group's, which takes 16 of them at a time. `tiles`, those of the groups that can have rows: up to half of the SMs Small's CTAs are alone
    // with their K, beyond it they are as fast from 32 rows on. K 7168, rows spread evenly / all in one group, here and on Small: 32 tiles (8 groups,
    // N 512) 64 rows 13.4 / 21.4 us and 29.5 / 29.9, 128 rows 13.4 / 40.5 and 29.6 / 30.1; 64 tiles (16 groups) 256 rows 23.3 / 79 and 29.8 / 30.3;
    // 128 tiles (32 groups) 32 rows 38 / 21 and 31 / 29, 64 rows 38 / 38 and 31 / 30, 256 rows 39 / 141 and 31 / 31.
    const int64_t n128 = (a.N + 127) / 128, tiles = std::min<int64_t>(a.groups, a.M) * n128;
    if (a.groups == 1 ? a.M <= 16 : rows <= 16 && a.groups * n128 < sms && a.M <= (2 * tiles <= sms ? 256 : 32)) return launch_int8_few(a, s);
    // 256 x 256: where 256 x 128 tiles take a second round of the pairs. 1000 rows 47 us and 59 on Pair, 512 rows, K 4096, 30 and 22; 16 groups of
    // 256 rows, K 2048, 73 and 77, 32 of 128 rows 93 and 89
    if (a.groups <= Large::kMaxGroups && rows >= 256 && ((a.M + 255) / 256) * n_tiles * 4 >= sms) return launch<Large, Out>(a, p, s);
    // 256 x 128 on pairs: where they give half of the pairs a tile (fewer are split over K on one-CTA tiles). 384 rows 32 us and 37 on Mid, 256
    // rows 32 and 25; 32 groups, K 2048: 64 rows each 63 and 84, 16 each 55 and 52 on Small
    const int64_t row_tiles = (a.M + 127) / 128 + (a.groups > 1 ? std::min<int64_t>(a.groups, a.M) / 2 : 0);
    if (rows > 16 && row_tiles * n_tiles * 4 >= sms) return launch<Pair, Out>(a, p, s);
    // 128 x 128 or 128 x 64: 100 rows 17 us and 22, 64 rows 18 and 15
    return rows > 64 ? launch<Mid, Out>(a, p, s) : launch<Small, Out>(a, p, s);
}

}  // namespace

size_t int8_matmul_workspace(int64_t, int64_t, int64_t, int) { return sizeof(int32_t) * kOpsHeaderInts; }

cudaError_t launch_int8_matmul(const moe_int8_matmul_args& a, void* workspace, cudaStream_t s) {
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
    p.kb_count = (int)((a.K + kStageK - 1) / kStageK);
    return a.out_type == MOE_TYPE_BF16 ? launch_out<__nv_bfloat16>(a, p, s) : launch_out<float>(a, p, s);
}

}  // namespace moe
