// The whole MoE layer for a few tokens in one cooperative launch (moe_layer in moe_ops.h):
//
//     y[t] = sum over the token's experts e of w[t,e] * (SiLU(x[t] W1g[e]) * (x[t] W1u[e])) W2[e]
//
// With few tokens every expert that is touched is multiplied by a handful of rows, so the time is that of reading its
// weights once. The kernel is a stream of weights through shared memory: one CTA per SM, a producer warp that keeps a ring
// of stages of 8 KB (BF16: 16 KB) full by TMA, and eight warps that multiply each stage by the tokens' rows with mma.sync
// (16 weight rows x 8 tokens x 16 of K), which at this shape is far from the tensor pipe's bound. The weight addresses
// depend on the routes alone, so the producer runs ahead across units, experts and from the first product into the
// second, while the consumers wait for activations.
//
// Phases:
//   1. router: every CTA takes its experts' dot products with all tokens in fp32, its warps on parts of H (CUDA cores: the
//      selection compares these sums); one CTA per token also rounds x to the f16 operand of the FP8 and FP4 formats. Grid barrier.
//   2. selection: each CTA selects for all tokens itself (up to 8 tokens), or for its share of them and a second barrier.
//      Each CTA then lists the experts with rows and their rows in shared memory.
//   3. first product: units of 16 outputs (16 gate and 16 up rows of W1; BF16: 64 and 64) of one expert. Each warp (BF16: pair
//      of warps) takes every eighth (fourth) stage whole, so that a stage costs one wait and one arrival and its latencies have the
//      time of eight stages; the warps' sums of a unit meet in shared memory, where one of two epilogue warps adds them up. SwiGLU of
//      them goes to the workspace in fp32 with the row's largest magnitude. A counter per expert says when its rows are complete.
//   4. second product: units of 32 hidden columns (BF16: 128) of one expert, expert by expert, over all of K or a part of it. The
//      slots' sums go to the workspace; the epilogue warp that brings the last ones of a column group adds its tokens' slots up
//      in order.
// Units are handed out one by one from a counter, a few ahead of the producer: equal shares of the bytes left the SMs up to a sixth
// apart at the end. What a unit computes does not depend on who computes it, and there are no atomics on values: results do not
// depend on timing.
//
// Operands. BF16: x as it is; the activations as two bf16 (hi + lo, 16 bits of them) and two MMAs. FP8 and FP4: the weights are
// exact in f16, x and the activations are scaled by a power of two of their row to below 2^15 and rounded once to f16: 11 bits, and
// below 2^-14 multiples of 2^-24. So bf16 x is exact down to 2^-31 of its row's maximum and rounded to multiples of 2^-38 of it at
// worst below; activations lose up to 2^-11 a value, against 2^-8 of the bf16 result. The FP8 weight scale multiplies the fp32
// sum over each 64 of K; the UE8M0 scales of FP4 multiply the f16 codes relative to the largest of the four blocks that a stage's
// sum covers (exact while they lie within 2^36 of it) and that one the fp32 sum.
//
// Bound by HBM where a call reads much of few experts. Fractions are of the measured copy rate and count the weights of the experts
// that the routes in fact touched. 3 tokens, top-2 of 8 experts, 4096 / 14336, BF16: 1.41 GB (4 experts) in 228 us, 0.93; 1.76 GB (5)
// in 274, 0.96; 2.11 GB (6) in 320, 0.99. 32 tokens, top-8 of 256 experts in the best 4 of 8 groups and a shared one, hidden 7168,
// intermediate 2048, FP8: 6.08 GB (138 experts) in 1.11-1.12 ms, 0.81. One token of the same: 397 MB (9) in 82 us, 0.72 (13 us are
// the router and the selection, whose barriers and latencies no weights hide). 5 tokens, top-6 of 64, 2048 / 768, FP4: 58 MB (23) in
// 53-58 us, by inputs and machine. With more column tiles an expert, and in FP4, it is not HBM (what it is was not profiled): BF16,
// 8 experts as above, 16 / 32 / 64 tokens 464 / 666 / 1267 us (0.91, 0.63, 0.33); FP4, top-8 of 128 and a shared one, 4096 / 1536,
// 5 / 16 / 32 / 64 tokens 169 / 390 / 584 / 986 us (0.30, 0.31, 0.29, 0.19; that of 33-64 tokens spills some 460 bytes a thread);
// FP8 of that layer, 4 / 16 / 64 tokens 110 / 310 / 706 us (0.75, 0.73, 0.51), 104 for 4 with the routes given.
//
// Every wait is bounded (2 s): MOE_ERR_TIMEOUT. From then on the CTA's waits end at once, no slot of the ring is handed back for
// another copy, its queue of units ends, and it passes the barriers that are left.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "gate_select.cuh"
#include "layer_parts.h"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace layer {

using namespace tc;

constexpr int kWarps = 8;                       // consumers
constexpr int kAllWarps = 12;                   // warp 8 is the producer, 9 and 10 the epilogue, 11 fetches units
constexpr int kThreads = 32 * kAllWarps;
// registers of warps 8-11 and of the consumers from phase 3 on: 128 * 104 + 256 * 200 = 384 * 168, what the launch holds
constexpr int kLaunchRegs = 168, kFewRegs = 104, kManyRegs = 200;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kMaxT = MOE_LAYER_MAX_TOKENS;
constexpr int kMaxSlots = kMaxT * 32;
constexpr int kEpiWarps = 2;                    // warps 9 and 10 take the sums of a unit further
constexpr int kMaxE = 1024;

// Stage geometry. K-contiguous formats: two boxes of 32 rows x 128 bytes. BF16: 64 of K x two boxes of 64 columns. All boxes
// have the 128-byte swizzle (the 16-byte unit u of line r is at u ^ (r % 8)). A warp multiplies a stage in four slices of K.
template <int kFmt>
struct Geo {
    static constexpr bool kBf16 = kFmt == MOE_LAYER_BF16;
    static constexpr bool kFp4 = kFmt == MOE_LAYER_FP4_MX;
    static constexpr int kRows = kBf16 ? 128 : 32;  // weight rows of a unit
    static constexpr int kOut1 = kRows / 2;         // outputs of a unit of the first product
    static constexpr int kStepK = kBf16 ? 64 : kFp4 ? 512 : 256;
    static constexpr int kSlices = 4, kSliceK = kStepK / kSlices;
    static constexpr int kStageBytes = kBf16 ? 16384 : 8192;
    static constexpr int kStages = kBf16 ? 8 : 16;
    static constexpr int kGroups = kBf16 ? 4 : 8;   // consumer groups: stage i is group i % kGroups's
    // a slot of the ring is always the same group's: two groups may be more than a use of the slot apart, and a wait for a
    // phase's parity cannot tell it from the phase two before
    static_assert(kStages % kGroups == 0, "slots and groups");
    static constexpr int kGroupWarps = kWarps / kGroups;
    static constexpr int kMt = kBf16 ? 4 : 2;       // 16-row MMA tiles of a warp
    static constexpr int kRedCol = kRows + 4;       // floats of a column of partial sums (two columns apart: 8 banks)
    static constexpr int kRedGroup = 8 * kRedCol;
    static constexpr int kRed = kGroups * kRedGroup + 8;  // and the inverse scale of each column's activations
    static constexpr int kReds = kBf16 ? 2 : 4;     // sets of partial sums on their way to the epilogue
    static_assert(kReds % kEpiWarps == 0, "likewise for the sets and the epilogue's warps, which take them in turn");
    // shared memory: ring | sets of partial sums | tables
    static constexpr int kRedOff = kStages * kStageBytes;
    static constexpr int kTabOff = kRedOff + kReds * 4 * kRed;
};

constexpr int kMaxBars = 48;
constexpr int kProducers = 4;                   // producer lanes, each on every fourth stage of the CTA's sequence
// Units are published up to kLead past the one that the producer's first lane is in. Its lanes go on together, from one stage each to
// the next, and a unit has at least one stage: the last lane needs the unit kProducers - 1 further at most, which is there without
// the first lane's help (with units of no stage it would wait for the first lane, and that for it).
constexpr int kLead = 3;
static_assert(kLead >= kProducers - 1, "units in reach of every producer lane");
// Units between the fetching warp and the slowest reader: kLead, one a stage of the ring (16) and one a set of partial sums (4, a unit
// has at least one) at most, and the ones being worked on.
constexpr int kQueue = 64;
constexpr uint32_t kNoUnit = 0xffffffffu;

struct Tables {
    uint64_t bars[kMaxBars];
    volatile uint64_t queue[kQueue];      // the CTA's units: (k + 1) << 32 | unit of the k-th
    volatile int begun;                   // units the producer has begun
    int n_active, last, abort;
    int count[kMaxE];
    int16_t expert[kMaxE];                // active experts
    int16_t start[kMaxE + 2];             // where their rows begin in row[]
    uint16_t row[kMaxSlots];              // slot = token * (K + S) + k
    uint8_t token[kMaxSlots];             // by slot
    float weight[kMaxSlots];              // by slot
    int16_t id[kMaxSlots];                // by slot, -1: none
};

struct Args {
    const uint16_t* x;
    const void* router;
    const void *w1, *w2;
    const void *s1, *s2;
    const float* bias;
    int32_t* ids_io;
    float* weights_io;
    uint16_t* y;
    moe_gate_options gate;
    int router_bf16;
    int T, H, I, E, K, S;
    float clamp;
    int splits;        // parts of K that a column group of an expert is cut into in the second product (layer_parts)
    int32_t* hdr;      // [0] error word, [1] barrier, [2] CTAs finished, [3] units handed out
    int32_t* dep;      // per active expert: finished column tiles of its units of the first product
    int32_t* cols;     // per column group: finished column tiles of the second product
    uint32_t* amax;    // per slot: largest |activation| so far, as bits
    float* logits;     // [T][E]
    int32_t* ids;      // [T][K]
    float* weights;    // [T][K]
    uint16_t* x16;     // f16 [T][H]
    float* xinv;       // [T]
    float* act;        // [slots][I]
    float* comb;       // [splits][slots][H]
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// the two e4m3 codes of half i of a word -> two f16 (exact)
template <int i>
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t word) {
    uint32_t r;
    asm("{\n\t.reg .b16 h0, h1;\n\tmov.b32 {h0, h1}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h%2;\n\t}" : "=r"(r) : "r"(word), "n"(i));
    return r;
}
// the two e2m1 codes of byte i -> two f16 (exact), low nibble first
template <int i>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t word) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}" : "=r"(r) : "r"(word), "n"(i));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 2^(kFp4Up - d) as f16 twice (d >= 0; 0 below the smallest subnormal). kFp4Up: as far up as the largest e2m1 value, 6, stays finite, so
// that the codes of blocks with smaller scales have the room below. The rows' inverse scales take it back (kFp4Down).
constexpr int kFp4Up = 13;
constexpr float kFp4Down = 1.0f / (1 << kFp4Up);
__device__ __forceinline__ uint32_t pow2_f16x2(int d) {
    const uint32_t h = d <= 14 + kFp4Up ? (uint32_t)(15 + kFp4Up - d) << 10 : d <= 24 + kFp4Up ? 1u << (24 + kFp4Up - d) : 0u;
    return h | (h << 16);
}
// The power of two that takes magnitudes up to `top` (bits) below 2^15, and its inverse. Zero, infinities and NaNs: 1.
__device__ __forceinline__ float row_scale(uint32_t top, float* inverse) {
    int e = (int)(top >> 23);
    if (top == 0u || e == 255) e = 141;
    e = max(e, 15);
    *inverse = __uint_as_float((uint32_t)(e - 14) << 23);     // 2^(e - 141)
    return __uint_as_float((uint32_t)(268 - e) << 23);        // 2^(141 - e)
}

// All CTAs have arrived n times (n counts the barriers of this launch); one thread waits, bounded.
__device__ __forceinline__ void grid_barrier(const Args& p, int n, volatile int* abort_flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(p.hdr + 1, 1);
        wait_count(p.hdr + 1, n * (int)gridDim.x, p.hdr, abort_flag);
        __threadfence();
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------
// phase 1: the router product
// ---------------------------------------------------------------------------------------

// Adds the products of one 16-byte vector of x with 8 router values.
__device__ __forceinline__ float dot8(uint4 w, const float (&r)[8], float sum) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(__uint_as_float(u[i] << 16), r[2 * i], sum);
        sum = fmaf(__uint_as_float(u[i] & 0xffff0000u), r[2 * i + 1], sum);
    }
    return sum;
}

__device__ __forceinline__ void router_values(const Args& p, int e, int v, float (&r)[8]) {
    if (p.router_bf16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.router) + (int64_t)e * p.H) + v);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = __uint_as_float(u[i] << 16);
            r[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.router) + (int64_t)e * p.H) + 2 * v;
        const float4 a = __ldg(q), b = __ldg(q + 1);
        r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    }
}

// The CTA's experts (two at a time: they share the reads of x), all warps on parts of H, 8 tokens at a time. parts: shared
// memory of kAllWarps * 16 floats.
static __device__ void router_phase(const Args& p, float* parts, int warp, int lane) {
    const int vecs = p.H / 8, grid = (int)gridDim.x;
    for (int e0 = blockIdx.x; e0 < p.E; e0 += 2 * grid) {
        const int e1 = e0 + grid;
        const bool two = e1 < p.E;
        for (int t0 = 0; t0 < p.T; t0 += 8) {
            const int nt = min(8, p.T - t0);
            float s0[8], s1[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s0[j] = s1[j] = 0.0f;
            for (int v = warp * 32 + lane; v < vecs; v += 32 * kAllWarps) {
                uint4 w[8];
                float r0[8], r1[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < nt) w[j] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + j) * p.H) + v);
                router_values(p, e0, v, r0);
                router_values(p, two ? e1 : e0, v, r1);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < nt) {
                        s0[j] = dot8(w[j], r0, s0[j]);
                        s1[j] = dot8(w[j], r1, s1[j]);
                    }
            }
            __syncthreads();  // the parts of the tokens before have been read
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < nt) {
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1) {
                        s0[j] += __shfl_xor_sync(0xffffffffu, s0[j], d);
                        s1[j] += __shfl_xor_sync(0xffffffffu, s1[j], d);
                    }
                    if (lane == 0) {
                        parts[warp * 16 + j] = s0[j];
                        parts[warp * 16 + 8 + j] = s1[j];
                    }
                }
            __syncthreads();
            const int j = threadIdx.x & 7, which = threadIdx.x >> 3;
            if (which < (two ? 2 : 1) && j < nt) {
                float s = 0.0f;
                for (int i = 0; i < kAllWarps; ++i) s += parts[i * 16 + which * 8 + j];
                p.logits[(int64_t)(t0 + j) * p.E + (which ? e1 : e0)] = s;
            }
        }
    }
}

// x of one token as f16, scaled by a power of two (all threads of the CTA); down: a factor of the inverse scale.
static __device__ void round_x(const Args& p, int t, float down, uint32_t* scratch) {
    const uint4* src = reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.H);
    uint32_t top = 0;
    for (int v = threadIdx.x; v < p.H / 8; v += kThreads) {
        const uint4 w = __ldg(src + v);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(u[i] & 0x7fff0000u, (u[i] << 16) & 0x7fff0000u));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAllWarps; ++i) top = max(top, scratch[i]);
    float inverse;
    const float s = row_scale(top, &inverse);
    uint4* dst = reinterpret_cast<uint4*>(p.x16 + (int64_t)t * p.H);
    for (int v = threadIdx.x; v < p.H / 8; v += kThreads) {
        const uint4 w = __ldg(src + v);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_f16(__uint_as_float(u[i] << 16) * s, __uint_as_float(u[i] & 0xffff0000u) * s);
        dst[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (threadIdx.x == 0) p.xinv[t] = inverse * down;
}

// ---------------------------------------------------------------------------------------
// phase 2: selection and the list of experts
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ void select_token(const Args& p, int t, float* scratch, int lane, int32_t* ids, float* weights) {
#pragma unroll 8
    for (int e = lane; e < p.E; e += 32) scratch[e] = __ldcg(p.logits + (int64_t)t * p.E + e);
    if (p.bias)
#pragma unroll 8
        for (int e = lane; e < p.E; e += 32) scratch[p.E + e] = __ldg(p.bias + e);
    gate_token(scratch, p.bias != nullptr, p.gate, p.E, p.K, lane, ids, weights);
}

// ids and weights (of the routed slots) -> the experts with rows, in order, and their rows. distinct: a token's ids are (as
// selected ones are).
static __device__ void list_experts(const Args& p, Tables& tb, const int32_t* ids, const float* weights, bool distinct) {
    const int Kt = p.K + p.S, Et = p.E + p.S, slots = p.T * Kt;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < Et; e += kThreads) tb.count[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const int t = s / Kt, k = s - t * Kt;
        int e = p.E + k - p.K;
        float w = 1.0f;
        if (k < p.K) {
            const int32_t* id = ids + t * p.K;
            const float* wt = weights + t * p.K;
            e = id[k];
            w = wt[k];
            if (e < -1 || e >= p.E) {
                record_error(p.hdr, MOE_ERR_BAD_ROUTE);
                e = -1;
            }
            if (!distinct && e >= 0) {  // an expert named twice by a token: one row with the sum of the weights
                bool first = true;
                for (int i = 0; i < p.K; ++i)
                    if (i != k && id[i] == e) {
                        if (i < k) first = false;
                        else w += wt[i];
                    }
                if (!first) e = -1;
            }
        }
        tb.id[s] = (int16_t)e;
        tb.token[s] = (uint8_t)t;
        tb.weight[s] = w;
        if (e >= 0) atomicAdd(&tb.count[e], 1);
    }
    __syncthreads();
    // running numbers of the experts with rows and of the rows, 32 experts a warp
    int n[3], rows[3], active[3], chunks = 0;  // of this warp's chunks (at most 1024 + 31 experts over 12 warps)
    __shared__ int chunk_rows[33], chunk_active[33];
    for (int c = warp; c * 32 < Et; c += kAllWarps, ++chunks) {
        const int e = c * 32 + lane;
        const int v = e < Et ? tb.count[e] : 0;
        int sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        const uint32_t on = __ballot_sync(0xffffffffu, v > 0);
        n[chunks] = v;
        rows[chunks] = sum - v;
        active[chunks] = __popc(on & ((1u << lane) - 1u));
        if (lane == 31) {
            chunk_rows[c] = sum;
            chunk_active[c] = __popc(on);
        }
    }
    __syncthreads();
    chunks = 0;
    for (int c = warp; c * 32 < Et; c += kAllWarps, ++chunks) {
        int r = 0, a = 0;
        for (int i = 0; i < c; ++i) {
            r += chunk_rows[i];
            a += chunk_active[i];
        }
        const int e = c * 32 + lane;
        r += rows[chunks];
        a += active[chunks];
        if (n[chunks] > 0) {
            tb.expert[a] = (int16_t)e;
            tb.start[a] = (int16_t)r;
        }
        if (e < Et) tb.count[e] = r;  // the next free place
        if (c * 32 + 32 >= Et && lane == 31) {
            tb.n_active = a + (n[chunks] > 0);
            tb.start[tb.n_active] = (int16_t)(r + n[chunks]);
        }
    }
    __syncthreads();
    // place within the expert in any order: rows are independent of each other
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const int e = tb.id[s];
        if (e >= 0) tb.row[atomicAdd(&tb.count[e], 1)] = (uint16_t)s;
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------
// phases 3 and 4
// ---------------------------------------------------------------------------------------

// The launch's work in units, handed out one by one: first those of the first product, expert by expert, then those of the second.
// A unit of the first is kOut1 outputs of an expert; of the second it is kRows hidden columns of an expert, over all of K or one
// of `splits` parts of it.
template <int kFmt>
struct Work {
    uint32_t per1, per2, n1, total;  // units per expert, of the first product, in all
    int steps1, steps2, split_steps;
    uint32_t splits;
    __device__ Work(const Args& p, int active) {
        using G = Geo<kFmt>;
        splits = p.splits;
        per1 = p.I / G::kOut1;
        per2 = p.H / G::kRows * splits;
        n1 = per1 * active;
        total = n1 + per2 * active;
        steps1 = (p.H + G::kStepK - 1) / G::kStepK;
        steps2 = (p.I + G::kStepK - 1) / G::kStepK;
        split_steps = part_steps(steps2, p.splits);
    }
};

struct Unit {
    int a, group, split, st0, st1;  // active expert; group of rows (or of hidden columns); part of K; stages [st0, st1)
};
template <int kFmt>
__device__ __forceinline__ Unit unit_first(const Work<kFmt>& wk, uint32_t u) {
    const uint32_t a = u / wk.per1;
    return {(int)a, (int)(u - a * wk.per1), 0, 0, wk.steps1};
}
template <int kFmt>
__device__ __forceinline__ Unit unit_second(const Work<kFmt>& wk, uint32_t u) {
    u -= wk.n1;
    const uint32_t a = u / wk.per2, r = u - a * wk.per2, g = r / wk.splits, q = r - g * wk.splits;
    const int st0 = (int)q * wk.split_steps;
    return {(int)a, (int)g, (int)q, st0, min(wk.steps2, st0 + wk.split_steps)};
}

// The CTA's k-th unit, kNoUnit after the last one. Every lane of every warp gets the same answer, also when the CTA gives up: an
// entry is written once, and fetch ends the sequence within its own limit, so this one, four times as long, is not reached. (Looking
// at the abort flag here let lanes part that have to stay together; a vote on the answer took 0.4 to 0.8 % of the layer's time.)
__device__ __forceinline__ uint32_t take(const Tables& tb, int k, int32_t* hdr, volatile int* abort_flag) {
    const volatile uint64_t* q = tb.queue + k % kQueue;
    uint64_t v = *q;
    if ((uint32_t)(v >> 32) == (uint32_t)k + 1u) return (uint32_t)v;
    const uint64_t t0 = globaltimer_ns();
    for (int i = 1;; ++i) {
        v = *q;
        if ((uint32_t)(v >> 32) == (uint32_t)k + 1u) return (uint32_t)v;
        if (i % 256 == 0 && globaltimer_ns() - t0 > 4 * kWaitTimeoutNs) {
            record_error(hdr, MOE_ERR_TIMEOUT);
            *abort_flag = 1;
            return kNoUnit;
        }
    }
}

// One lane: gets the CTA's units from the launch's counter, a few ahead of the producer, until they run out or the CTA gives up.
// Either way the last entry says so.
template <int kFmt>
__device__ __forceinline__ void fetch(const Args& p, Tables& tb, const Work<kFmt>& wk, volatile int* abort_flag) {
    uint32_t u = blockIdx.x;  // the first one is given
    for (int k = 0;; ++k) {
        bool end = u >= wk.total;
        if (k > 0) {
            const uint64_t t0 = globaltimer_ns();
            while (tb.begun + kLead < k) {
                if (*abort_flag || globaltimer_ns() - t0 > kWaitTimeoutNs) {
                    if (!*abort_flag) record_error(p.hdr, MOE_ERR_TIMEOUT);
                    *abort_flag = 1;
                    end = true;
                    break;
                }
                __nanosleep(32);
            }
            if (!end) {
                u = gridDim.x + (uint32_t)atomicAdd(p.hdr + 3, 1);
                end = u >= wk.total;
            }
        }
        tb.queue[k % kQueue] = ((uint64_t)(k + 1) << 32) | (end ? kNoUnit : u);
        if (end) return;
    }
}

template <int kFmt>
struct Ring {
    static_assert(2 * (Geo<kFmt>::kStages + Geo<kFmt>::kReds) <= kMaxBars, "barriers");
    uint32_t base, bars;
    int it = 0;
    __device__ uint32_t full(int s) const { return bars + 8u * s; }
    __device__ uint32_t empty(int s) const { return bars + 8u * (Geo<kFmt>::kStages + s); }
    // sets of partial sums: written by all consumers; read by the epilogue
    __device__ uint32_t red_full(int s) const { return bars + 8u * (2 * Geo<kFmt>::kStages + s); }
    __device__ uint32_t red_empty(int s) const { return bars + 8u * (2 * Geo<kFmt>::kStages + Geo<kFmt>::kReds + s); }
};

// The producer warp: four lanes take every fourth stage of the CTA's sequence each, so that the latencies of a stage's wait and
// of its barrier's byte count (some 150 cycles each) are those of four stages.
template <int kFmt>
__device__ __forceinline__ void produce(const Args& p, const CUtensorMap* map1, const CUtensorMap* map2, const Ring<kFmt>& ring,
                                        Tables& tb, const Work<kFmt>& wk, int lane, volatile int* abort_flag) {
    using G = Geo<kFmt>;
    static_assert(G::kStages % kProducers == 0, "a slot of the ring is always the same lane's");
    constexpr uint32_t kLanes = (1u << kProducers) - 1u;
    int k = 0, last = -1;                 // units taken; the last stage this lane issued
    uint32_t u = take(tb, k, p.hdr, abort_flag);
    bool second = u >= wk.n1;
    Unit un = {};
    if (u != kNoUnit) un = second ? unit_second(wk, u) : unit_first(wk, u);
    int it = lane, st = lane;             // this lane's stage: of the sequence, and of the unit past its first stage
    for (;; it += kProducers, st += kProducers) {
        while (u != kNoUnit && st >= un.st1 - un.st0) {
            st -= un.st1 - un.st0;
            u = take(tb, ++k, p.hdr, abort_flag);
            if (lane == 0) tb.begun = k;
            second = u >= wk.n1;
            if (u != kNoUnit) un = second ? unit_second(wk, u) : unit_first(wk, u);
        }
        if (__all_sync(kLanes, u == kNoUnit)) break;
        if (u != kNoUnit) {
            const int expert = tb.expert[un.a], r0 = un.group * (second ? G::kRows : G::kOut1), sti = un.st0 + st;
            const int s = it % G::kStages;
            const uint32_t dst = ring.base + (uint32_t)(s * G::kStageBytes), bar = ring.full(s);
            const CUtensorMap* map = second ? map2 : map1;
            if (mbar_wait(ring.empty(s), ((uint32_t)(it / G::kStages) & 1u) ^ 1u, p.hdr, abort_flag)) {
                if constexpr (G::kBf16) {
                    mbar_arrive_expect_tx(bar, 16384);
                    const int y = expert * (second ? p.I : p.H) + sti * 64;
                    tma_load_2d(dst, map, r0, y, bar);
                    tma_load_2d(dst + 8192, map, second ? r0 + 64 : p.I + r0, y, bar);
                } else {
                    const int row_bytes = (second ? p.I : p.H) / (G::kFp4 ? 2 : 1);
                    const int row = expert * (second ? p.H : 2 * p.I) + r0, x = sti * 256;
                    const bool two = x + 128 < row_bytes;  // a box that ends inside a row is filled up with zeros
                    mbar_arrive_expect_tx(bar, two ? 8192u : 4096u);
                    // first product: 16 gate rows, then the up rows of the same outputs (the map's third coordinate)
                    if (second) tma_load_2d(dst, map, x, row, bar);
                    else tma_load_3d(dst, map, x, row, 0, bar);
                    if (two) {
                        if (second) tma_load_2d(dst + 4096, map, x + 128, row, bar);
                        else tma_load_3d(dst + 4096, map, x + 128, row, 0, bar);
                    }
                }
                last = it;
            } else {
                u = kNoUnit;  // gave up: what is in flight is waited for below
            }
        }
        __syncwarp(kLanes);
    }
    // drain: every copy this lane issued has landed (bounded)
    for (int j = last; j >= 0 && j > last - G::kStages; j -= kProducers)
        if (!mbar_drain(ring.full(j % G::kStages), (uint32_t)(j / G::kStages) & 1u, p.hdr)) break;
}

// MMA rows g and g + 8 of 16-row tile m are the stage's rows 8 m + perm(g) and 16 + 8 m + perm(g): lanes 4 g .. 4 g + 3 read 64
// bytes of a row, and the rows of two neighbouring g, four apart, lie in different halves of the swizzled lines.
__device__ __forceinline__ int perm(int g) { return (g >> 1) | ((g & 1) << 2); }

// One column tile's values for a slice: B words as they are in memory (fp32 activations: two to a word of B).
template <int kFmt, bool kSecond>
struct Columns {
    using G = Geo<kFmt>;
    static constexpr int kB = G::kBf16 ? 2 : G::kFp4 ? 16 : 8;  // 16-bit pairs of the tile
    static constexpr int kWords = kSecond ? 2 * kB : kB;
    static constexpr int kBytes = kSecond ? 4 : 2;              // of a value in memory
    uint32_t w[kWords];

    // The x row or activation row `row` (-1: none), from this lane's first value of a slice on.
    static __device__ __forceinline__ const uint8_t* base(const Args& p, int row, int lane) {
        if (row < 0) return nullptr;
        const uint8_t* q = kSecond ? reinterpret_cast<const uint8_t*>(p.act + (int64_t)row * p.I)
                                   : reinterpret_cast<const uint8_t*>((G::kBf16 ? p.x : p.x16) + (int64_t)row * p.H);
        return q + kBytes * (lane & 3) * (G::kBf16 ? 2 : G::kFp4 ? 32 : 16);
    }
    __device__ __forceinline__ void load(const uint8_t* q, int k) {
        const bool on = q != nullptr;
        q += kBytes * k;
        if constexpr (G::kBf16) {
            if constexpr (kSecond) {
                const uint2 u = on ? *reinterpret_cast<const uint2*>(q) : make_uint2(0, 0);
                const uint2 v = on ? *reinterpret_cast<const uint2*>(q + 32) : make_uint2(0, 0);
                w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
            } else {
                w[0] = on ? *reinterpret_cast<const uint32_t*>(q) : 0u;
                w[1] = on ? *reinterpret_cast<const uint32_t*>(q + 16) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = on ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0, 0, 0, 0);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
    }
};

// The weight scales of a slice. FP8: of the unit's two 128-row blocks (gate, up). FP4: four bytes, one for each 32 of K, of the
// rows g and g + 8 of both 16-row tiles.
template <int kFmt, bool kSecond>
struct Scales {
    using G = Geo<kFmt>;
    uint32_t s[G::kFp4 ? 4 : 2];
    static __device__ __forceinline__ const uint8_t* base(const Args& p, int expert, int r0, int lane) {
        const int K = kSecond ? p.I : p.H, N = kSecond ? p.H : 2 * p.I;
        const uint8_t* q = static_cast<const uint8_t*>(kSecond ? p.s2 : p.s1);
        if constexpr (G::kFp4) return q + ((int64_t)expert * N + r0 + perm(lane >> 2)) * (K / 32);
        else if constexpr (!G::kBf16) return q + 4 * ((int64_t)expert * (N / 128) + r0 / 128) * (K / 128);
        else return nullptr;
    }
    __device__ __forceinline__ void load(const Args& p, const uint8_t* q, int k) {
        const int K = kSecond ? p.I : p.H;
        if constexpr (G::kFp4) {
            q += k / 32;
#pragma unroll
            for (int i = 0; i < 4; ++i)  // i = 2 m: tile m's row g, 2 m + 1: its row g + 8
                s[i] = __ldg(reinterpret_cast<const uint32_t*>(q + (int64_t)((i >> 1) * 8 + ((i & 1) ? (kSecond ? 16 : p.I) : 0)) * (K / 32)));
        } else if constexpr (!G::kBf16) {
            q += 4 * (k / 128);
            s[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
            s[1] = kSecond ? s[0] : __ldg(reinterpret_cast<const uint32_t*>(q + (int64_t)4 * (p.I / 128) * (K / 128)));
        }
    }
};

// The weights of a warp's slice of a stage as MMA operands and their products with the column tiles, added to acc. The first
// tile's values are there (most experts have no more than its 8 rows), the others' are loaded here.
template <int kFmt, bool kSecond, int NT>
__device__ __forceinline__ void multiply_slice(const Args& p, uint32_t stage, int slice, int k, const Columns<kFmt, kSecond>& first,
                                               const Scales<kFmt, kSecond>& sc, const int (&rows)[NT], const float (&ascale)[NT],
                                               int tiles, int warp, int lane, float (&acc)[Geo<kFmt>::kMt][NT][4]) {
    using G = Geo<kFmt>;
    using Cols = Columns<kFmt, kSecond>;
    constexpr int kMmas = Cols::kB / 2;
    uint32_t a[G::kMt][kMmas][4];
    float f0[G::kMt], f1[G::kMt];  // scales of the sums of rows g and g + 8
#pragma unroll
    for (int m = 0; m < G::kMt; ++m) {
        f0[m] = f1[m] = 1.0f;
        if constexpr (G::kBf16) {
            // [K row][64 columns] boxes: lane l gives row l % 8 (+ 8 for matrices 2, 3) and columns + 8 for 1, 3
            const int krow = slice * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, c8 = (lane >> 3) & 1;
            ldmatrix_x4_trans(a[m][0], stage + (uint32_t)((warp & 1) * 8192 + krow * 128 + (((2 * m + c8) ^ (krow & 7)) << 4)));
        } else {
            const int r = m * 8 + perm(lane >> 2), unit = (slice & 1) * 4 + (lane & 3);
            const uint32_t at = stage + (uint32_t)((slice >> 1) * 4096 + r * 128 + ((unit ^ (r & 7)) << 4));
            const uint4 u = lds128(at), v = lds128(at + 16 * 128);  // rows g and g + 8 of the tile
            const uint32_t ug[4] = {u.x, u.y, u.z, u.w}, vg[4] = {v.x, v.y, v.z, v.w};
            if constexpr (G::kFp4) {
                // this lane's codes relative to the largest scale of the four blocks
                auto most = [](uint32_t w) { return max(max(w & 255u, (w >> 8) & 255u), max((w >> 16) & 255u, w >> 24)); };
                const uint32_t w0 = sc.s[2 * m], w1 = sc.s[2 * m + 1], m0 = most(w0), m1 = most(w1);
                const uint32_t p0 = pow2_f16x2((int)(m0 - ((w0 >> (8 * (lane & 3))) & 255u)));
                const uint32_t p1 = pow2_f16x2((int)(m1 - ((w1 >> (8 * (lane & 3))) & 255u)));
                f0[m] = ue8m0_to_float((uint8_t)m0);
                f1[m] = ue8m0_to_float((uint8_t)m1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[m][2 * q][0] = mul_f16x2(e2m1x2_f16x2<0>(ug[q]), p0);
                    a[m][2 * q][1] = mul_f16x2(e2m1x2_f16x2<0>(vg[q]), p1);
                    a[m][2 * q][2] = mul_f16x2(e2m1x2_f16x2<1>(ug[q]), p0);
                    a[m][2 * q][3] = mul_f16x2(e2m1x2_f16x2<1>(vg[q]), p1);
                    a[m][2 * q + 1][0] = mul_f16x2(e2m1x2_f16x2<2>(ug[q]), p0);
                    a[m][2 * q + 1][1] = mul_f16x2(e2m1x2_f16x2<2>(vg[q]), p1);
                    a[m][2 * q + 1][2] = mul_f16x2(e2m1x2_f16x2<3>(ug[q]), p0);
                    a[m][2 * q + 1][3] = mul_f16x2(e2m1x2_f16x2<3>(vg[q]), p1);
                }
            } else {
                f0[m] = __uint_as_float(sc.s[0]);
                f1[m] = __uint_as_float(sc.s[1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[m][q][0] = e4m3x2_f16x2<0>(ug[q]);
                    a[m][q][1] = e4m3x2_f16x2<0>(vg[q]);
                    a[m][q][2] = e4m3x2_f16x2<1>(ug[q]);
                    a[m][q][3] = e4m3x2_f16x2<1>(vg[q]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n >= tiles) break;
        Cols c;
        if (n == 0) c = first;
        else c.load(Cols::base(p, rows[n], lane), k);
        if constexpr (G::kBf16) {
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (kSecond) {
                    const float u = __uint_as_float(c.w[2 * i]), v = __uint_as_float(c.w[2 * i + 1]);
                    hi[i] = pack_bf16(u, v);
                    // an infinity or NaN stays in the high part alone
                    const float du = u - __uint_as_float(hi[i] << 16), dv = v - __uint_as_float(hi[i] & 0xffff0000u);
                    lo[i] = pack_bf16(fabsf(u) < INFINITY ? du : 0.0f, fabsf(v) < INFINITY ? dv : 0.0f);
                } else {
                    hi[i] = c.w[i];
                }
            }
#pragma unroll
            for (int m = 0; m < G::kMt; ++m) {
                mma_bf16(acc[m][n], a[m][0], hi[0], hi[1]);
                if constexpr (kSecond) mma_bf16(acc[m][n], a[m][0], lo[0], lo[1]);
            }
        } else {
            uint32_t bw[Cols::kB];
#pragma unroll
            for (int i = 0; i < Cols::kB; ++i) {
                if constexpr (kSecond)
                    bw[i] = pack_f16(__uint_as_float(c.w[2 * i]) * ascale[n], __uint_as_float(c.w[2 * i + 1]) * ascale[n]);
                else
                    bw[i] = c.w[i];
            }
#pragma unroll
            for (int m = 0; m < G::kMt; ++m) {
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < kMmas; ++j) mma_f16(part, a[m][j], bw[2 * j], bw[2 * j + 1]);
                acc[m][n][0] = fmaf(part[0], f0[m], acc[m][n][0]);
                acc[m][n][1] = fmaf(part[1], f0[m], acc[m][n][1]);
                acc[m][n][2] = fmaf(part[2], f1[m], acc[m][n][2]);
                acc[m][n][3] = fmaf(part[3], f1[m], acc[m][n][3]);
            }
        }
    }
}

// Waits for the rows of active expert a, those of the next ones looked at together: experts below `known` have theirs
// (units come expert by expert).
__device__ __forceinline__ void wait_rows(const Args& p, const Tables& tb, int a, int per1, int& known, int lane,
                                          volatile int* abort_flag) {
    if (a < known) return;
    // a unit counts its column tiles
    auto target = [&](int e) { return per1 * ((tb.start[e + 1] - tb.start[e] + 7) / 8); };
    const bool on = a + lane < tb.n_active;
    const uint32_t there = __ballot_sync(0xffffffffu, on && ld_acquire_gpu(p.dep + a + lane) >= target(on ? a + lane : a));
    const int ready = there == 0xffffffffu ? 32 : __ffs(~there) - 1;
    known = a + max(ready, 1);
    if (ready == 0 && lane == 0) wait_count(p.dep + a, target(a), p.hdr, abort_flag);
    __syncwarp();  // the lanes' acquires order what the warp reads from here on
}

// The units of one product by a consumer warp, from the CTA's k-th (u) on: of each its group's stages (i % kGroups of the CTA's
// sequence) times the expert's rows, then its sums to the epilogue, one set a column tile. Groups without a stage of a unit only
// sign for their part of the sets. A stage's scales and first columns are asked for before the wait for the stage (asking for those of the next
// stage or unit while a slice is multiplied was measured slower: 1494 us instead of 1182 for 32 tokens and 256 experts).
template <int kFmt, bool kSecond, int NT>
__device__ __forceinline__ void consume(const Args& p, Ring<kFmt>& ring, int& set, int& k, uint32_t& u, float* reds,
                                        const Tables& tb, const Work<kFmt>& wk, int warp, int lane, volatile int* abort_flag) {
    using G = Geo<kFmt>;
    using Cols = Columns<kFmt, kSecond>;
    using Sc = Scales<kFmt, kSecond>;
    constexpr int kSlices = G::kSlices;
    // so many slices of the first tile's values are held, as far as registers go
    constexpr int kSums = G::kMt * 4 * NT;
    constexpr int kAhead = 4 * Cols::kWords + kSums <= 80 ? 4 : 2 * Cols::kWords + kSums <= 80 ? 2 : 1;
    const int K = kSecond ? p.I : p.H, group = warp / G::kGroupWarps;
    int seq = ring.it, known = 0;  // number of the unit's first stage in the CTA's sequence; see wait_rows

    Cols cols[kAhead];
    Sc sc[kSlices];
    for (; u != kNoUnit && (kSecond || u < wk.n1); u = take(tb, ++k, p.hdr, abort_flag)) {
        const Unit un = kSecond ? unit_second(wk, u) : unit_first(wk, u);
        const int a = un.a, r0 = un.group * (kSecond ? G::kRows : G::kOut1), st0 = un.st0, st1 = un.st1;
        int st = st0 + (group - seq % G::kGroups + G::kGroups) % G::kGroups;  // the group's first stage of the unit
        const bool part = st < st1;
        if (kSecond) wait_rows(p, tb, a, (int)wk.per1, known, lane, abort_flag);
        const int begin = tb.start[a], n_rows = tb.start[a + 1] - begin, tiles = (n_rows + 7) / 8;
        float acc[G::kMt][NT][4], ainv[NT];
        if (part) {
            int rows[NT];  // of this lane's column of each tile; -1 past the expert's rows
            float ascale[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int c = n * 8 + (lane >> 2);
                rows[n] = -1;
                ascale[n] = ainv[n] = 1.0f;
                if (c < n_rows) {
                    const int slot = tb.row[begin + c];
                    rows[n] = kSecond ? slot : (int)tb.token[slot];
                    if constexpr (kSecond && !G::kBf16) ascale[n] = row_scale(__ldcg(p.amax + slot), &ainv[n]);
                }
            }
            const uint8_t *col = Cols::base(p, rows[0], lane), *scale = Sc::base(p, tb.expert[a], r0, lane);
#pragma unroll
            for (int m = 0; m < G::kMt; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.0f;
            for (; st < st1; st += G::kGroups) {
                const int it = seq + st - st0, s = it % G::kStages, k0 = st * G::kStepK;
#pragma unroll
                for (int j = 0; j < kSlices; ++j)
                    if (k0 + j * G::kSliceK < K) {
                        sc[j].load(p, scale, k0 + j * G::kSliceK);
                        if (j < kAhead) cols[j].load(col, k0 + j * G::kSliceK);
                    }
                // a wait that ran out is the warp's last: the slot is not handed back, as the copy into it may still be under way
                if (!__all_sync(0xffffffffu, mbar_wait(ring.full(s), (uint32_t)(it / G::kStages) & 1u, p.hdr, abort_flag))) {
                    u = kNoUnit;
                    return;
                }
                const uint32_t stage = ring.base + (uint32_t)(s * G::kStageBytes);
#pragma unroll
                for (int j = 0; j < kSlices; ++j) {
                    if (k0 + j * G::kSliceK < K)
                        multiply_slice<kFmt, kSecond, NT>(p, stage, j, k0 + j * G::kSliceK, cols[j % kAhead], sc[j], rows, ascale, tiles,
                                                          warp, lane, acc);
                    if (j + kAhead < kSlices && k0 + (j + kAhead) * G::kSliceK < K) cols[j % kAhead].load(col, k0 + (j + kAhead) * G::kSliceK);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(ring.empty(s));
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n, ++set) {
            if (n >= tiles) break;
            const int q = set % G::kReds;
            mbar_wait(ring.red_empty(q), ((uint32_t)(set / G::kReds) & 1u) ^ 1u, p.hdr, abort_flag);
            if (part) {
                float* dst = reds + q * G::kRed + group * G::kRedGroup + (G::kBf16 ? (warp & 1) * 64 : 0);
                const int g = lane >> 2, t = lane & 3;
#pragma unroll
                for (int m = 0; m < G::kMt; ++m) {
                    const int r = G::kBf16 ? m * 16 + g : m * 8 + perm(g), r8 = G::kBf16 ? r + 8 : r + 16;
                    dst[(2 * t) * G::kRedCol + r] = acc[m][n][0];
                    dst[(2 * t + 1) * G::kRedCol + r] = acc[m][n][1];
                    dst[(2 * t) * G::kRedCol + r8] = acc[m][n][2];
                    dst[(2 * t + 1) * G::kRedCol + r8] = acc[m][n][3];
                }
                // once per set: by the group that holds the unit's first stage
                if (kSecond && !G::kBf16 && seq % G::kGroups == group && t == 0)
                    reds[(q + 1) * G::kRed - 8 + g] = G::kFp4 ? ainv[n] * kFp4Down : ainv[n];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.red_full(q));
        }
        seq += st1 - st0;
    }
    ring.it = seq;
}

// The sum of the groups' parts of one value of a set; the unit's stages begin at `it` and are `steps` many. In the order of the
// stages, whichever groups they fell to: the sum does not depend on what the CTA did before.
template <int kFmt>
__device__ __forceinline__ float red_sum(const float* red, int it, int steps, int col, int row) {
    using G = Geo<kFmt>;
    const float* q = red + col * G::kRedCol + row;
    float s = 0.0f;
    if (steps >= G::kGroups) {
#pragma unroll
        for (int i = 0; i < G::kGroups; ++i) s += q[(it + i) % G::kGroups * G::kRedGroup];
    } else {
        for (int i = 0; i < steps; ++i) s += q[(it + i) % G::kGroups * G::kRedGroup];
    }
    return s;
}

// A unit of the first product by epilogue warp w, which takes every second set: SwiGLU of its outputs and the rows' largest
// magnitudes.
template <int kFmt>
__device__ __forceinline__ void finish_first(const Args& p, Ring<kFmt>& ring, int& set, const float* reds, const Tables& tb, int a,
                                             int r0, int w, int lane, volatile int* abort_flag) {
    using G = Geo<kFmt>;
    const int begin = tb.start[a], n_rows = tb.start[a + 1] - begin;
    const int steps = (p.H + G::kStepK - 1) / G::kStepK, tiles = (n_rows + 7) / 8;
    int mine = 0;
    for (int n = 0; n < tiles; ++n, ++set) {
        if (set % kEpiWarps != w) continue;
        ++mine;
        const int q = set % G::kReds;
        const float* red = reds + q * G::kRed;
        // FP8, FP4: 16 outputs of two columns at a time; BF16: 64 of one, two a lane
        constexpr int kCols = G::kBf16 ? 1 : 2, kEach = G::kBf16 ? 2 : 1;
        float inv[8 / kCols];
#pragma unroll
        for (int i = 0; i < 8 / kCols; ++i) {
            const int c = n * 8 + i * kCols + (G::kBf16 ? 0 : lane >> 4);
            inv[i] = !G::kBf16 && c < n_rows ? __ldcg(p.xinv + tb.token[tb.row[begin + c]]) : 1.0f;
        }
        mbar_wait(ring.red_full(q), (uint32_t)(set / G::kReds) & 1u, p.hdr, abort_flag);
#pragma unroll
        for (int i = 0; i < 8 / kCols; ++i) {
            const int cc = i * kCols + (G::kBf16 ? 0 : lane >> 4), c = n * 8 + cc;
            if (c < n_rows) {
                const int slot = tb.row[begin + c];
#pragma unroll
                for (int h = 0; h < kEach; ++h) {
                    const int j = G::kBf16 ? h * 32 + lane : lane & 15;
                    const float g = red_sum<kFmt>(red, ring.it, steps, cc, j) * inv[i];
                    const float u = red_sum<kFmt>(red, ring.it, steps, cc, G::kOut1 + j) * inv[i];
                    const float v = swiglu1(g, u, p.clamp);
                    p.act[(int64_t)slot * p.I + r0 + j] = v;
                    if constexpr (!G::kBf16) {
                        const uint32_t top = __reduce_max_sync(0xffffu << (lane & 16), __float_as_uint(v) & 0x7fffffffu);
                        if ((lane & 15) == 0) atomicMax(p.amax + slot, top);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.red_empty(q));
    }
    if (mine && lane == 0) {
        __threadfence();
        atomicAdd(p.dep + a, mine);
    }
    ring.it += steps;
}

// The tokens' sums over their slots of one column group (a warp): weights times the parts of K, in order, to bf16. Eight loads in
// flight: this is what the last units of a launch wait for.
template <int kFmt>
__device__ __forceinline__ void combine(const Args& p, const Tables& tb, int group, int lane) {
    using G = Geo<kFmt>;
    constexpr int kPerToken = G::kRows / 4, kBatch = 8;  // lanes of a token: four columns each
    const int Kt = p.K + p.S, n = Kt * p.splits;
    const int64_t part = (int64_t)p.T * Kt * p.H;
    for (int t = lane / kPerToken; t < p.T; t += 32 / kPerToken) {
        const int64_t at = (int64_t)group * G::kRows + lane % kPerToken * 4;
        const float* row = p.comb + (int64_t)t * Kt * p.H + at;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int k = 0, q = 0;  // slot and part of the next load
        for (int j = 0; j < n; j += kBatch) {
            float4 v[kBatch];
            float w[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int slot = t * Kt + k;
                const bool on = j + i < n && tb.id[min(slot, kMaxSlots - 1)] >= 0;
                w[i] = on ? tb.weight[slot] : 0.0f;
                v[i] = on ? __ldcg(reinterpret_cast<const float4*>(row + (int64_t)k * p.H + q * part)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (++q == p.splits) {
                    q = 0;
                    ++k;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                y.x = fmaf(w[i], v[i].x, y.x), y.y = fmaf(w[i], v[i].y, y.y), y.z = fmaf(w[i], v[i].z, y.z), y.w = fmaf(w[i], v[i].w, y.w);
        }
        *reinterpret_cast<uint2*>(p.y + (int64_t)t * p.H + at) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
}

// A unit of the second product by epilogue warp w: the sums of its sets to the slots' rows in the workspace. The warp with the last
// of a column group's `total` sets (all experts, all parts) adds the tokens' rows up.
template <int kFmt>
__device__ __forceinline__ void finish_second(const Args& p, Ring<kFmt>& ring, int& set, const float* reds, const Tables& tb,
                                              const Unit& un, int total, int w, int lane, volatile int* abort_flag) {
    using G = Geo<kFmt>;
    const int begin = tb.start[un.a], n_rows = tb.start[un.a + 1] - begin, tiles = (n_rows + 7) / 8, steps = un.st1 - un.st0;
    const int slots = p.T * (p.K + p.S);
    float* out = p.comb + (int64_t)un.split * slots * p.H + (int64_t)un.group * G::kRows;
    int mine = 0;
    for (int n = 0; n < tiles; ++n, ++set) {
        if (set % kEpiWarps != w) continue;
        ++mine;
        const int q = set % G::kReds;
        const float* red = reds + q * G::kRed;
        mbar_wait(ring.red_full(q), (uint32_t)(set / G::kReds) & 1u, p.hdr, abort_flag);
#pragma unroll
        for (int cc = 0; cc < 8; ++cc) {
            const int c = n * 8 + cc;
            if (c >= n_rows) break;
            const float f = G::kBf16 ? 1.0f : red[G::kRed - 8 + cc];
            float* dst = out + (int64_t)tb.row[begin + c] * p.H;
#pragma unroll
            for (int h = 0; h < G::kRows / 32; ++h) dst[h * 32 + lane] = red_sum<kFmt>(red, ring.it, steps, cc, h * 32 + lane) * f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.red_empty(q));
    }
    ring.it += steps;
    if (!mine) return;
    int done = 0;
    if (lane == 0) {
        __threadfence();
        done = atomicAdd(p.cols + un.group, mine) + mine;
    }
    done = __shfl_sync(0xffffffffu, done, 0);
    if (done == total) {
        __threadfence();
        combine<kFmt>(p, tb, un.group, lane);
        if (lane == 0) p.cols[un.group] = 0;
    }
}

// NT: column tiles that an expert can have (T <= 8 NT).
template <int kFmt, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    layer_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2,
                 const __grid_constant__ Args p) {
    using G = Geo<kFmt>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    Tables& tb = *reinterpret_cast<Tables*>(smem + G::kTabOff);
    float* reds = reinterpret_cast<float*>(smem + G::kRedOff);
    volatile int* abort_flag = &tb.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ring<kFmt> ring;
    ring.base = base;
    ring.bars = smem_u32(tb.bars);
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(ring.full(s), 1);
            mbar_init(ring.empty(s), G::kGroupWarps);
        }
        for (int s = 0; s < G::kReds; ++s) {
            mbar_init(ring.red_full(s), kWarps);
            mbar_init(ring.red_empty(s), 1);
        }
        tb.abort = 0;
        tb.begun = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < kQueue) tb.queue[threadIdx.x] = 0;
    __syncthreads();

    // ---- phase 1
    int barriers = 0;
    if (p.router) router_phase(p, reds, warp, lane);
    if constexpr (!G::kBf16)
        for (int t = (int)gridDim.x - 1 - (int)blockIdx.x; t < p.T; t += gridDim.x)
            round_x(p, t, G::kFp4 ? kFp4Down : 1.0f, reinterpret_cast<uint32_t*>(reds));
    if (p.router || !G::kBf16) grid_barrier(p, ++barriers, abort_flag);

    // ---- phase 2
    const int32_t* ids = p.ids_io;
    const float* weights = p.weights_io;
    if (p.router) {
        const bool all = p.T <= kWarps;  // every CTA selects for all tokens
        int32_t* to_ids = all ? reinterpret_cast<int32_t*>(reds) : p.ids;
        float* to_w = all ? reds + kWarps * 32 : p.weights;
        float* scratch = reinterpret_cast<float*>(smem) + warp * gate_scratch(kMaxE);
        const int t0 = all ? warp : (int)blockIdx.x + warp * (int)gridDim.x;
        if (warp < kWarps && t0 < p.T) select_token(p, t0, scratch, lane, to_ids + t0 * p.K, to_w + t0 * p.K);
        if (all) __syncthreads();
        else grid_barrier(p, ++barriers, abort_flag);
        ids = to_ids;
        weights = to_w;
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < p.T * p.K; i += kThreads) {
                if (p.ids_io) p.ids_io[i] = ids[i];
                if (p.weights_io) p.weights_io[i] = weights[i];
            }
    }
    list_experts(p, tb, ids, weights, p.router != nullptr);
    // the ring's memory was scratch until here: ordered before the copies that fill it
    fence_proxy_async_smem();
    __syncthreads();
    const Work<kFmt> wk(p, tb.n_active);

    // ---- phases 3 and 4
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == kWarps) {
            if (lane < kProducers) produce<kFmt>(p, &map1, &map2, ring, tb, wk, lane, abort_flag);
        } else if (warp <= kWarps + kEpiWarps) {
            // the sets alternate between the two warps: each has the time of two for a unit's fence and counter
            const int w = warp - kWarps - 1;
            int total = 0;  // sets of a column group of the second product
            for (int a = lane; a < tb.n_active; a += 32) total += (tb.start[a + 1] - tb.start[a] + 7) / 8;
            total = (int)__reduce_add_sync(0xffffffffu, (uint32_t)total) * p.splits;
            int set = 0, k = 0;
            uint32_t u = take(tb, 0, p.hdr, abort_flag);
            for (; u < wk.n1; u = take(tb, ++k, p.hdr, abort_flag)) {
                const Unit un = unit_first(wk, u);
                finish_first<kFmt>(p, ring, set, reds, tb, un.a, un.group * G::kOut1, w, lane, abort_flag);
            }
            for (; u != kNoUnit; u = take(tb, ++k, p.hdr, abort_flag))
                finish_second<kFmt>(p, ring, set, reds, tb, unit_second(wk, u), total, w, lane, abort_flag);
        } else if (lane == 0) {
            fetch<kFmt>(p, tb, wk, abort_flag);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        int set = 0, k = 0;
        uint32_t u = take(tb, 0, p.hdr, abort_flag);
        consume<kFmt, false, NT>(p, ring, set, k, u, reds, tb, wk, warp, lane, abort_flag);
        consume<kFmt, true, NT>(p, ring, set, k, u, reds, tb, wk, warp, lane, abort_flag);
    }
    if (tb.n_active == 0)
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)p.T * p.H; i += (int64_t)gridDim.x * kThreads)
            p.y[i] = 0;

    // ---- the last CTA leaves the counters at zero
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        tb.last = atomicInc(reinterpret_cast<unsigned*>(p.hdr) + 2, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (tb.last) {
        for (int i = threadIdx.x; i < tb.n_active; i += kThreads) p.dep[i] = 0;
        for (int i = threadIdx.x; i < p.T * (p.K + p.S); i += kThreads) p.amax[i] = 0u;
        if (threadIdx.x == 0) p.hdr[1] = p.hdr[3] = 0;
    }
}

template <int kFmt>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)Geo<kFmt>::kTabOff + sizeof(Tables);
}

template <int kFmt, int NT>
cudaError_t launch_tiles(const Args& p, cudaStream_t s) {
    static_assert(smem_bytes<kFmt>() <= 232448, "shared memory");
    int device = 0;
    const cudaError_t err = once_per_device(&device, [](int) {
        const cudaError_t e = cudaFuncSetAttribute(layer_kernel<kFmt, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<kFmt>());
        return e != cudaSuccess ? e : check_register_split(reinterpret_cast<const void*>(layer_kernel<kFmt, NT>), kLaunchRegs);
    });
    if (err != cudaSuccess) return err;
    CUtensorMap m1 = {}, m2 = {};
    if constexpr (kFmt == MOE_LAYER_BF16) {
        const uint64_t Et = (uint64_t)p.E + p.S;
        if (!tc_make_map_2d(&m1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.w1, 2 * (uint64_t)p.I, Et * p.H, 64, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B) ||
            !tc_make_map_2d(&m2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.w2, (uint64_t)p.H, Et * p.I, 64, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    } else {
        const uint64_t Et = (uint64_t)p.E + p.S, half = kFmt == MOE_LAYER_FP4_MX ? 2 : 1;
        const uint64_t b1 = p.H / half, b2 = p.I / half;  // bytes of a row
        // W1 as [gate or up][row][bytes]: a box takes 16 rows of each
        const uint64_t d1[3] = {b1, Et * 2 * p.I - p.I, 2}, s1[2] = {b1, b1 * p.I};
        const uint32_t box1[3] = {128, 16, 2};
        const uint64_t d2[2] = {b2, Et * p.H}, s2[1] = {b2};
        const uint32_t box2[2] = {128, 32};
        if (!tc_make_map_nd(&m1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.w1, d1, s1, box1, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !tc_make_map_nd(&m2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.w2, d2, s2, box2, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tc_num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<kFmt>();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another: all of them are resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_kernel<kFmt, NT>, m1, m2, p);
}

// Instantiated per format in translation units of their own (moe_layer_*.cu).
template <int kFmt>
cudaError_t launch_fmt(const Args& p, cudaStream_t s) {
    if (p.T <= 8) return launch_tiles<kFmt, 1>(p, s);
    if (p.T <= 16) return launch_tiles<kFmt, 2>(p, s);
    if (p.T <= 32) return launch_tiles<kFmt, 4>(p, s);
    return launch_tiles<kFmt, 8>(p, s);
}

}  // namespace layer

}  // namespace moe
