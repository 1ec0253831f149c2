// Rows in the order of their experts (moe_permute in moe_ops.h): a stable counting sort of the T*K slots by expert, then a copy of each
// token's row to its K rows.
//
// Sort. The row of a slot is (slots of lower experts) + (earlier slots of its expert), which fixes the order without atomics
// whose order could change it: counts may be added up in any order, ranks are taken in the order of the slots.
//   - few slots: one launch in which every CTA has a token, counts all ids for itself (shared memory) and copies its row.
//   - more: the slots in up to 128 runs, a CTA each. One launch counts the runs' experts; in a second every CTA adds up the runs before its own,
//     counts its warps' parts and ranks 32 slots at a time with match.any; a third copies and clears
//     the counts.
//
// Bound by HBM's writes: a token is read once and written K times. 8192 x 8 x 7168 bf16 (1.06 GB): 169 us, 6.26 TB/s, 0.93 of the copy
// rate, where a fill alone runs at 4.0 TB/s; 9 us of them sort (a cluster of eight CTAs that exchanged its totals took 16).
// 7 x 8 x 7168 codes: 4.5 us on the device, the chain of ids, counts and copies.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

// Slots up to which one launch does it all, and tokens x slots, the ids that its CTAs count together. bf16, one launch and three, H 1024 / 7168:
// 512 x 8 6.7 / 14.1 and 10.8 / 16.4 us, 1024 x 4 8.6 / 16.2 and 9.5 / 16.2, 512 x 16 11.2 / 35.1 and 12.6 / 27.4; 2048 x 1 7.7 / 10.9 and 9.0 /
// 12.7, 2896 x 1 12.5 / 17.4 and 9.4 / 15.3, 4096 x 1 19.2 / 27.3 and 10.3 / 23.9, 2048 x 2 11.0 / 18.2 and 9.6 / 17.3.
constexpr int64_t kFewSlots = 4096, kFewIds = int64_t(1) << 22;
inline bool few_slots(int64_t T, int64_t K) { return T * K <= kFewSlots && T * T * K <= kFewIds; }

constexpr int kFewThreads = 256;
constexpr int kSortWarps = 32, kSortThreads = 32 * kSortWarps;
// Runs of slots that are sorted by a CTA each, and slots of one: every CTA reads all runs' counts (65536 slots of 256 experts, rows of 16 bytes: 128
// runs of 512 16.9 us, 64 of 1024 14.3, 16 of 4096 16.0; 4.2 million slots 237 us with 128 runs, 287 with 64, before the counts were cleared: 239).
constexpr int kMaxRuns = 128, kMinRun = 1024;
constexpr int kCopyWarps = 8;
constexpr int kCopyVecs = 4;  // vectors of a lane on their way at a time

struct SortArgs {
    const int32_t* ids;
    int32_t *offsets, *row_src, *slot_row, *hdr;
    int32_t* counts;  // [run][expert]
    int n, E, K;
    int run, runs;    // slots of a run (whole groups of 32), and their number
};

struct CopyArgs {
    const uint8_t* x;
    uint8_t* rows;
    const float* scale;
    float* row_scale;
    const int32_t* slot_row;
    int64_t bytes, x_stride, rows_stride;  // bytes of a row and between rows
    int32_t* counts;                       // the runs' counts, and how many there are
    int T, K, scales, segments, num_counts;
};

// expert of a slot, -1 without one; ids that name no expert are reported
__device__ __forceinline__ int slot_expert(const SortArgs& p, int s) {
    const int e = __ldg(p.ids + s);
    if (e >= 0 && e < p.E) return e;
    if (e != -1) record_error(p.hdr, MOE_ERR_BAD_ROUTE);
    return -1;
}

template <int V>
struct Vec;
template <>
struct Vec<16> { using type = uint4; };
template <>
struct Vec<8> { using type = uint2; };
template <>
struct Vec<4> { using type = uint32_t; };
template <>
struct Vec<2> { using type = uint16_t; };
template <>
struct Vec<1> { using type = uint8_t; };

// One warp copies vectors [v0, v1) of token t's row to the rows of its slots; `row`: lane k holds slot k's row or -1.
template <int V>
__device__ __forceinline__ void copy_segment(const CopyArgs& p, int t, int row, int64_t v0, int64_t v1, int lane) {
    using W = typename Vec<V>::type;
    const W* src = reinterpret_cast<const W*>(p.x + (int64_t)t * p.x_stride);
    for (int64_t v = v0 + lane; v - lane < v1; v += 32 * kCopyVecs) {
        W w[kCopyVecs];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j)
            if (v + 32 * j < v1) w[j] = __ldg(src + v + 32 * j);
        for (int k = 0; k < p.K; ++k) {
            const int r = __shfl_sync(0xffffffffu, row, k);
            if (r < 0) continue;
            W* dst = reinterpret_cast<W*>(p.rows + (int64_t)r * p.rows_stride);
#pragma unroll
            for (int j = 0; j < kCopyVecs; ++j)
                if (v + 32 * j < v1) dst[v + 32 * j] = w[j];
        }
    }
}

__device__ __forceinline__ void copy_scales(const CopyArgs& p, int t, int row, int lane) {
    for (int k = 0; k < p.K; ++k) {
        const int r = __shfl_sync(0xffffffffu, row, k);
        if (r < 0) continue;
        for (int i = lane; i < p.scales; i += 32) p.row_scale[(int64_t)r * p.scales + i] = __ldg(p.scale + (int64_t)t * p.scales + i);
    }
}

// CTA t < T: token t; CTA T: the offsets and the ends of row_src.
template <int V>
__global__ void __launch_bounds__(kFewThreads) permute_few_kernel(SortArgs p, CopyArgs c) {
    __shared__ int all[kRowExperts], before[kRowExperts];  // slots of each expert, those ahead of this token
    __shared__ int my_row[kRowTopk];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.E; e += kFewThreads) all[e] = before[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < p.n; s += kFewThreads) {
        const int e = slot_expert(p, s);
        if (e < 0) continue;
        atomicAdd(&all[e], 1);
        if (s < t * p.K) atomicAdd(&before[e], 1);
    }
    __syncthreads();
    if (t == c.T) {
        if (warp != 0) return;
        int carry = 0;
        for (int b = 0; b < p.E; b += 32) {
            int v = b + lane < p.E ? all[b + lane] : 0;
            const int own = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (b + lane < p.E) p.offsets[b + lane] = carry + v - own;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) p.offsets[p.E] = carry;
        for (int r = carry + lane; r < p.n; r += 32) p.row_src[r] = -1;
        return;
    }
    // slot k of the token: one warp adds up the lower experts' slots
    for (int k = warp; k < p.K; k += kFewThreads / 32) {
        const int id = lane < p.K ? slot_expert(p, t * p.K + lane) : -1;
        const int e = __shfl_sync(0xffffffffu, id, k);
        int sum = 0;
        for (int i = lane; i < e; i += 32) sum += all[i];
        sum = __reduce_add_sync(0xffffffffu, sum);
        const int twice = __popc(__ballot_sync(0xffffffffu, id == e && lane < k));  // the same expert at an earlier k
        if (lane == 0) {
            const int row = e < 0 ? -1 : sum + before[e] + twice;
            my_row[k] = row;
            p.slot_row[t * p.K + k] = row;
            if (row >= 0) p.row_src[row] = t * p.K + k;
        }
    }
    __syncthreads();
    const int row = lane < p.K ? my_row[lane] : -1;
    const int64_t vecs = c.bytes / V, part = ((vecs + 31) / 32 + kFewThreads / 32 - 1) / (kFewThreads / 32) * 32;
    copy_segment<V>(c, t, row, min(vecs, warp * part), min(vecs, (warp + 1) * part), lane);
    if (c.scale && warp == 0) copy_scales(c, t, row, lane);
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(SortArgs p) {
    __shared__ int count[kRowExperts];
    if (threadIdx.x < p.E) count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t s1 = min((int64_t)p.n, (int64_t)(blockIdx.x + 1) * p.run);
#pragma unroll 4
    for (int64_t s = (int64_t)blockIdx.x * p.run + threadIdx.x; s < s1; s += kSortThreads) {
        const int e = slot_expert(p, (int)s);
        if (e >= 0) atomicAdd(count + e, 1);
    }
    __syncthreads();
    if (threadIdx.x < p.E) p.counts[(int64_t)blockIdx.x * p.E + threadIdx.x] = count[threadIdx.x];
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(SortArgs p) {
    extern __shared__ int hist[];  // [warp][expert]: the warp's slots of the expert, then where the next of them goes
    __shared__ int all[kRowExperts], lower[kRowExperts];  // slots of the expert, and those of the runs before
    __shared__ int warp_sum[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    if (e < p.E) all[e] = lower[e] = 0;
    for (int i = threadIdx.x; i < kSortWarps * p.E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    // the threads share the runs where there are fewer experts than threads
    const int parts = kSortThreads / p.E, part = threadIdx.x / p.E, at = threadIdx.x - part * p.E;
    if (part < parts) {
        int sum = 0, before = 0;
#pragma unroll 16
        for (int r = part; r < p.runs; r += parts) {
            const int v = __ldg(p.counts + (int64_t)r * p.E + at);
            sum += v;
            if (r < (int)blockIdx.x) before += v;
        }
        if (sum) atomicAdd(all + at, sum);
        if (before) atomicAdd(lower + at, before);
    }
    // parts of a run: whole groups of 32 slots
    const int per = (p.run / 32 + kSortWarps - 1) / kSortWarps * 32;
    const int64_t end = min((int64_t)p.n, (int64_t)(blockIdx.x + 1) * p.run);
    const int64_t s0 = min(end, (int64_t)blockIdx.x * p.run + warp * per), s1 = min(end, s0 + per);
    int* mine = hist + warp * p.E;
#pragma unroll 4
    for (int64_t s = s0 + lane; s < s1; s += 32) {
        const int id = slot_expert(p, (int)s);
        if (id >= 0) atomicAdd(mine + id, 1);
    }
    __syncthreads();
    const int own = e < p.E ? all[e] : 0;
    int scan = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += u;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int ahead = 0, routed = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int v = warp_sum[w];
        if (w < warp) ahead += v;
        routed += v;
    }
    const int first = ahead + scan - own;
    if (blockIdx.x == 0) {
        if (e < p.E) p.offsets[e] = first;
        if (e == 0) p.offsets[p.E] = routed;
    }
    if (e < p.E) {
        int next = first + lower[e];
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int v = hist[w * p.E + e];
            hist[w * p.E + e] = next;
            next += v;
        }
    }
    __syncthreads();
    for (int64_t s = s0 + lane; s - lane < s1; s += 32) {
        const int id = s < s1 ? slot_expert(p, (int)s) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int row = id >= 0 ? mine[id] + rank : -1;
        __syncwarp();
        if (id >= 0 && rank == 0) mine[id] += __popc(same);
        __syncwarp();
        if (s < s1) p.slot_row[s] = row;
        if (row >= 0) p.row_src[row] = (int)s;
    }
    for (int64_t r = routed + (int64_t)blockIdx.x * kSortThreads + threadIdx.x; r < p.n; r += (int64_t)gridDim.x * kSortThreads) p.row_src[r] = -1;
}

template <int V>
__global__ void __launch_bounds__(32 * kCopyWarps) copy_kernel(CopyArgs c) {
    const int lane = threadIdx.x & 31;
    const int64_t vecs = c.bytes / V, items = (int64_t)c.T * c.segments;
    // the workspace goes back as zeros, which the next call on it may count on (other operators keep counters there)
    static_assert(kMaxRuns * kRowExperts <= 32 * kCopyWarps << 16, "the first 2^16 CTAs have all counts");
    if (blockIdx.x < 1u << 16)
        for (int i = blockIdx.x * (32 * kCopyWarps) + threadIdx.x; i < c.num_counts; i += min(gridDim.x, 1u << 16) * (32 * kCopyWarps)) c.counts[i] = 0;
    for (int64_t item = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); item < items; item += (int64_t)gridDim.x * kCopyWarps) {
        const int64_t t = item / c.segments, seg = item - t * c.segments, v0 = seg * (32 * kCopyVecs);
        const int row = lane < c.K ? __ldg(c.slot_row + t * c.K + lane) : -1;
        copy_segment<V>(c, (int)t, row, v0, min(vecs, v0 + 32 * kCopyVecs), lane);
        if (c.scale && seg == 0) copy_scales(c, (int)t, row, lane);
    }
}

template <int V>
cudaError_t launch_v(const SortArgs& p, CopyArgs c, cudaStream_t s) {
    if (few_slots(c.T, c.K)) {
        permute_few_kernel<V><<<c.T + 1, kFewThreads, 0, s>>>(p, c);
        return cudaGetLastError();
    }
    static_assert(sizeof(int) * kSortWarps * kRowExperts + 16384 <= 232448, "shared memory");
    int device = 0;
    const cudaError_t e = once_per_device(&device, [](int) {
        return cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(int) * kSortWarps * kRowExperts);
    });
    if (e != cudaSuccess) return e;
    count_kernel<<<p.runs, kSortThreads, 0, s>>>(p);
    place_kernel<<<p.runs, kSortThreads, sizeof(int) * kSortWarps * p.E, s>>>(p);
    const int64_t per_row = (c.bytes / V + 32 * kCopyVecs - 1) / (32 * kCopyVecs);
    c.segments = (int)per_row;
    c.counts = p.counts, c.num_counts = p.runs * p.E;
    const int64_t ctas = (c.T * per_row + kCopyWarps - 1) / kCopyWarps;
    copy_kernel<V><<<(unsigned)std::min<int64_t>(ctas, 0x7fffffff), 32 * kCopyWarps, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace

size_t permute_workspace(int64_t T, int K, int E) {
    return sizeof(int32_t) * (kOpsHeaderInts + (few_slots(T, K) ? 0 : (size_t)kMaxRuns * E));
}

cudaError_t launch_permute(const moe_permute_args& a, int T, int K, int E, int32_t* hdr, cudaStream_t s) {
    const int size = a.type == MOE_TYPE_F32 ? 4 : a.type == MOE_TYPE_BF16 ? 2 : 1;
    SortArgs p = {};
    p.ids = a.topk_ids;
    p.offsets = a.offsets, p.row_src = a.row_src, p.slot_row = a.slot_row;
    p.hdr = hdr, p.counts = hdr + kOpsHeaderInts;
    p.n = T * K, p.E = E, p.K = K;
    p.run = std::max(kMinRun, (p.n + kMaxRuns - 1) / kMaxRuns + 31) / 32 * 32;
    p.runs = (p.n + p.run - 1) / p.run;
    CopyArgs c = {};
    c.x = static_cast<const uint8_t*>(a.x);
    c.rows = static_cast<uint8_t*>(a.rows);
    c.scale = a.scales > 0 ? a.scale : nullptr;
    c.row_scale = a.row_scale;
    c.slot_row = a.slot_row;
    c.bytes = a.H * size, c.x_stride = a.x_stride * size, c.rows_stride = a.rows_stride * size;
    c.T = T, c.K = K, c.scales = a.scales;
    // the widest vector that every row starts and ends on
    const uint64_t low = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.rows) | (uint64_t)c.bytes |
                         (uint64_t)c.x_stride | (uint64_t)c.rows_stride;
    if (low % 16 == 0) return launch_v<16>(p, c, s);
    if (low % 8 == 0) return launch_v<8>(p, c, s);
    if (low % 4 == 0) return launch_v<4>(p, c, s);
    return low % 2 == 0 ? launch_v<2>(p, c, s) : launch_v<1>(p, c, s);
}

}  // namespace moe
