/*
 * moe_ops.h -- C ABI of the operators around the expert FFN of moe_ffn.h: the router, products of 8-bit
 * floating-point matrices with a scale for each block of 128, the whole MoE layer for a few tokens, rows sorted
 * by expert and back with their gradients, and products of 8-bit integer matrices with a scale for each row.
 *
 * The conventions of moe_ffn.h hold: plain device pointers and sizes, nothing allocated, asynchronous on
 * `stream`, argument errors found on the host before anything is launched. What differs:
 *   - Row strides are given where a matrix may be a part of a wider one (in elements; rows are contiguous).
 *   - The workspace of these operators is set to zero once by the caller, before its first use
 *     (moe_ops_workspace_init, or any memset): its counters are zero again at the end of every call, so no call
 *     pays for clearing them. Calls that may run at the same time need a workspace each. After a device-side
 *     error (moe_check_device_error; bounded waits that ran out) it is set to zero again before its next use.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of plain floating-point operands. */
typedef enum {
    MOE_TYPE_BF16 = 0,
    MOE_TYPE_F32 = 1,
    MOE_TYPE_CODES8 = 2 /* one byte an element, copied as it is (int8, e4m3 ..): moe_permute alone */
} moe_type;

/* Sets a workspace of this header's operators to zero. MOE_ERR_WORKSPACE: missing or not 256-byte aligned. */
MOE_API moe_status moe_ops_workspace_init(void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------------------------------------
 * The router
 * ------------------------------------------------------------------------------------------------------ */

typedef enum {
    MOE_SCORE_SOFTMAX = 0, /* s[e] = exp(l[e]) / sum over all E of exp(l)    */
    MOE_SCORE_SIGMOID = 1  /* s[e] = 1 / (1 + exp(-l[e]))                    */
} moe_score;

typedef struct {
    int32_t score;       /* a moe_score                                                                     */
    int32_t num_groups;  /* G in 1..32, a divisor of E: the experts in G equal runs                          */
    int32_t topk_groups; /* 1..G groups stay eligible; topk_groups * E/G >= K                                */
    int32_t group_top;   /* 1 or 2: a group's rank is the sum of its so many largest choice values           */
    int32_t normalize;   /* nonzero: the K weights are divided by (their sum + 1e-20)                        */
    float route_scale;   /* finite; multiplies the weights                                                   */
} moe_gate_options;

/* Expert ids and gate weights from router logits, in the form moe_plan, moe_forward and moe_layer take.
 *   choice value   c[e] = s[e] + bias[e] with a bias, else l[e] for softmax scores (same order as s, undisturbed
 *                  by rounding) and s[e] for sigmoid ones.
 *   selection      the topk_groups groups of highest rank, then the K experts of highest c among theirs, highest
 *                  first; equal values (of groups and of experts) go to the lowest index. A group is ranked by the
 *                  experts that are not masked: with fewer than group_top of them by their sum, with none below
 *                  every other group.
 *   weight         s[id] of the chosen ones (without the bias), normalised and scaled as the options say.
 *   masked experts a logit of -inf, or a NaN, is never chosen. When fewer than K experts are left in the groups that
 *                  stay, the remaining ids are -1 (moe_plan's masked route) and their weights 0. A finite logit,
 *                  the type's lowest value too, is a candidate like any other. A logit of +inf has s = 1 (softmax:
 *                  1 / the number of +inf logits of the row, and 0 for the finite ones). A bias of NaN masks its
 *                  expert too, one of -inf makes it the last candidate.
 *   logits         device [T,E] of `type`, row_stride >= E elements apart (T = d->num_tokens, E =
 *                  d->num_experts, K = d->topk; the other sizes in d are not read).
 *   bias           device fp32 [E] or NULL.      opt   NULL: softmax, one group, normalised, scale 1.
 *   topk_ids       device int32 [T,K];           topk_weights  device fp32 [T,K].
 * Scores are fp32. Errors: MOE_ERR_INVALID_ARG (sizes outside 1 <= K <= min(32, E), E <= 1024, T*K <= 2^24;
 * options outside the ranges above; a missing or misaligned pointer; row_stride < E). */
MOE_API moe_status moe_gate(const void* logits, moe_type type, int64_t row_stride, const float* bias,
                            const moe_gate_options* opt, const moe_dims* d, int32_t* topk_ids, float* topk_weights,
                            moe_stream_t stream);

/* ------------------------------------------------------------------------------------------------------
 * 8-bit floating point with a scale for each block of 128
 * ------------------------------------------------------------------------------------------------------ */

enum {
    MOE_QUANT_POW2 = 1u /* scales are powers of two: the smallest that is >= amax / 448, and 2^-126 at least */
};

/* Rows of x in e4m3 with an fp32 scale for each 128 columns (the last block may be smaller):
 *   s = amax / 448 (1 where that is 0), q = e4m3(x / s): fp32 IEEE division, round half to even.
 * A block that holds a NaN or an infinity gets a NaN or infinite scale, so products with it are not finite.
 *   x      device [rows, cols] of `type`, x_stride >= cols elements apart.
 *   q      device e4m3 [rows, cols], q_stride >= cols apart.
 *   scale  device fp32 [rows, ceil(cols/128)], contiguous.
 * Errors: MOE_ERR_INVALID_ARG (negative sizes, cols = 0 with rows > 0, short strides, a missing pointer, x or scale
 * not aligned to its elements, unknown flags). */
MOE_API moe_status moe_fp8_quantize(const void* x, moe_type type, int64_t rows, int64_t cols, int64_t x_stride, void* q,
                                    int64_t q_stride, float* scale, uint32_t flags, moe_stream_t stream);

/* out[m,n] = sum_kb a_scale[m,kb] * b_scale[g,n/128,kb] * sum_{k in block kb} a[m,k] * b[g,n,k]
 *   a        e4m3 [M,K], a_stride apart;   a_scale  fp32 [M, ceil(K/128)], contiguous
 *   b        e4m3 [groups][N,K], rows b_stride apart, groups N * b_stride apart
 *   b_scale  fp32 [groups][ceil(N/128), ceil(K/128)], contiguous
 *   offsets  NULL with groups = 1: every row of a is multiplied by b. Else device int32 [groups + 1], not
 *            decreasing, offsets[0] = 0 and offsets[groups] <= M (the offsets of moe_plan, for rows in plan order): rows
 *            [offsets[g], offsets[g+1]) are multiplied by b[g]. Rows from offsets[groups] on are not written. Values
 *            outside [0, M] are taken as the nearest bound, one below an earlier one as that one.
 *   out      bf16 or fp32 [M,N], out_stride apart
 * The sums over a block of K are the tensor core's fp32 sums, those over the blocks are fp32 fused multiply-adds with the
 * fp32 product of the two scales.
 * Limits: 0 <= M <= 2^31 - 512, 1 <= N <= 2^20, 16 <= K <= 2^20, 1 <= groups <= 1024, M * out_stride and the other
 * extents < 2^62; K, a_stride and b_stride multiples of 16, a and b 16-byte aligned (TMA); out aligned to its
 * elements. Errors: MOE_ERR_INVALID_ARG for these, MOE_ERR_WORKSPACE, MOE_ERR_CUDA. */
typedef struct {
    const void* a;
    const float* a_scale;
    const void* b;
    const float* b_scale;
    const int32_t* offsets;
    void* out;
    int64_t M, N, K;
    int64_t a_stride, b_stride, out_stride;
    int32_t groups;
    int32_t out_type; /* a moe_type */
} moe_fp8_matmul_args;

/* Bytes of workspace of moe_fp8_matmul for these sizes (0 when they are outside its limits); zeroed once. */
MOE_API size_t moe_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t groups);
MOE_API moe_status moe_fp8_matmul(const moe_fp8_matmul_args* args, void* workspace, size_t workspace_bytes,
                                  moe_stream_t stream);

/* ------------------------------------------------------------------------------------------------------
 * The whole layer for a few tokens
 * ------------------------------------------------------------------------------------------------------ */

/* Weight formats of moe_layer (x is bf16 in each; shared experts follow the E routed ones, as in moe_dims).
 *   MOE_LAYER_BF16       w1 bf16 [E+S,H,2I], w2 bf16 [E+S,I,H] (MOE_A16W16's weights)
 *   MOE_LAYER_FP8_BLOCK  w1 e4m3 [E+S,2I,H] + fp32 [E+S,2I/128,H/128], w2 e4m3 [E+S,H,I] + fp32 [E+S,H/128,I/128]
 *   MOE_LAYER_FP4_MX     MOE_A8W4_FP8_FP4's weights: e2m1 [E+S,2I,H/2] + UE8M0 [E+S,2I,H/32], and w2 likewise */
typedef enum {
    MOE_LAYER_BF16 = 0,
    MOE_LAYER_FP8_BLOCK = 1,
    MOE_LAYER_FP4_MX = 2
} moe_layer_weights;

enum {
    MOE_LAYER_MAX_TOKENS = 64
};

/* y[t] = sum_k w[t,k] FFN_{id[t,k]}(x[t]) + sum over shared experts s of FFN_s(x[t]),
 * FFN_e(x) = (SiLU(x W1g) * (x W1u)) W2, with ids and weights from the logits x . router^T as moe_gate has them.
 * One launch: the router product, the selection, both expert products and the combine.
 *   x            bf16 [T,H]
 *   router       bf16 or fp32 [E,H] (router_type), or NULL: topk_ids and topk_weights are inputs then, as
 *                moe_forward takes them (-1: masked route; other ids outside [0,E): MOE_ERR_BAD_ROUTE in the
 *                error word, the route skipped).
 *   gate, gate_bias  as moe_gate's opt and bias (not read without a router)
 *   topk_ids, topk_weights  int32 and fp32 [T,K]: outputs with a router (NULL: not wanted)
 *   y            bf16 [T,H]; a token with no route and no shared expert gets zeros
 * Weights are converted exactly to the 16-bit operands of the tensor cores (FP4: where the scales of each 128 of K of a row
 * lie within 2^36 of the largest of them; codes with smaller ones are rounded to multiples of 2^-37 times it); x, the
 * activations (rounded once to 16-bit halves that hold at least 11 bits of them) and all sums are described at the
 * kernel. Deterministic.
 * Limits: those of moe_dims (H and I multiples of 128), T <= MOE_LAYER_MAX_TOKENS (else MOE_ERR_UNSUPPORTED: use
 * moe_forward); all tensors contiguous and 16-byte aligned. */
typedef struct {
    const void* x;
    const void* router;
    moe_operand w1, w2;
    const moe_gate_options* gate;
    const float* gate_bias;
    int32_t* topk_ids;
    float* topk_weights;
    void* y;
    int32_t router_type;          /* a moe_type */
    int32_t weights;              /* a moe_layer_weights */
    uint32_t has_activation_clamp;
    float activation_clamp;       /* as in moe_options */
} moe_layer_args;

/* Bytes of workspace of moe_layer for up to d->num_tokens tokens, the other sizes as in d (0 when they are outside its
 * limits); zeroed once. */
MOE_API size_t moe_layer_workspace_bytes(const moe_dims* d, moe_layer_weights weights);
MOE_API moe_status moe_layer(const moe_layer_args* args, const moe_dims* d, void* workspace, size_t workspace_bytes,
                             moe_stream_t stream);

/* ------------------------------------------------------------------------------------------------------
 * Rows in the order of their experts, and back
 * ------------------------------------------------------------------------------------------------------ */

/* Sorts the T*K slots (token i, k-th expert: slot i*K+k) by expert, slots of one expert in ascending order, and copies
 * each slot's token to its row: rows[p] = x[row_src[p] / K] for p < R = offsets[E], the routed slots.
 *   topk_ids   device int32 [T,K]: -1 is a masked route (no row); other ids outside [0,E) have no row either and set
 *              MOE_ERR_BAD_ROUTE in the workspace's error word. An id may be there twice in a token.
 *   x          device [T,H] of `type`, x_stride elements apart;    rows  [T*K,H] of it, rows_stride apart
 *   scale      NULL, or device fp32 [T,scales], contiguous: goes to row_scale [T*K,scales] as x goes to rows
 *   offsets    device int32 [E+1]: expert e's rows are [offsets[e], offsets[e+1]) (what the grouped products take)
 *   row_src    device int32 [T*K]: the slot of row p, -1 for p >= R
 *   slot_row   device int32 [T*K]: the row of each slot, -1 without one (what moe_unpermute takes)
 * Rows from R on are not written; the outputs overlap no input. The order is fixed by the ids alone, unlike moe_plan's.
 * The gradient with respect to x is moe_unpermute of the rows' gradients, without weights. T = d->num_tokens, K = d->topk,
 * E = d->num_experts; the other sizes in d are not read. Errors: MOE_ERR_INVALID_ARG (sizes outside 1 <= K <= 32, 1 <= E <= 1024, T*K <= 2^24,
 * 1 <= H <= 2^30, 0 <= scales <= 2^20; short strides; a missing or misaligned pointer), MOE_ERR_WORKSPACE, MOE_ERR_CUDA. */
typedef struct {
    const void* x;
    const float* scale;
    const int32_t* topk_ids;
    void* rows;
    float* row_scale;
    int32_t* offsets;
    int32_t* row_src;
    int32_t* slot_row;
    int64_t H, x_stride, rows_stride;
    int32_t type;   /* a moe_type */
    int32_t scales; /* not read without a scale */
} moe_permute_args;

/* Bytes of workspace of moe_permute for up to d->num_tokens tokens (0 when T, K or E are outside its limits); zeroed once. */
MOE_API size_t moe_permute_workspace_bytes(const moe_dims* d);
MOE_API moe_status moe_permute(const moe_permute_args* args, const moe_dims* d, void* workspace, size_t workspace_bytes,
                               moe_stream_t stream);

/* y[i] = sum over k of topk_weights[i,k] * rows[slot_row[i,k]], in fp32 in the order of k and rounded once.
 *   rows          device [T*K,H] of `type` (bf16 or fp32), rows_stride elements apart
 *   slot_row      device int32 [T,K] of moe_permute: a slot whose entry is outside [0, T*K) adds nothing, whatever its
 *                 weight; a token without any other gets zeros. Rows that no slot names are not read.
 *   topk_weights  device fp32 [T,K], or NULL: 1 (the gradient of moe_permute)
 *   y             device [T,H] of y_type (bf16 or fp32), y_stride apart; no part of rows
 * Sizes, limits and errors as in moe_permute. */
MOE_API moe_status moe_unpermute(const void* rows, moe_type type, int64_t rows_stride, const int32_t* slot_row,
                                 const float* topk_weights, const moe_dims* d, int64_t H, void* y, moe_type y_type,
                                 int64_t y_stride, moe_stream_t stream);

/* Gradients of moe_unpermute from dy, that of y:
 *   d_rows[slot_row[i,k]] = topk_weights[i,k] * dy[i]           in fp32, rounded once to the rows' type
 *   d_weights[i,k]        = <rows[slot_row[i,k]], dy[i]>        in fp32; 0 for a slot without a row
 *   dy         device [T,H] of dy_type (bf16 or fp32), dy_stride apart
 *   rows       device [T*K,H] of `type`, rows_stride apart; not read (and may be NULL) without d_weights
 *   d_rows     device [T*K,H] of `type`, d_rows_stride apart; rows that no slot names are not written
 *   d_weights  device fp32 [T,K], or NULL: not wanted
 * slot_row and topk_weights as in moe_unpermute; no two slots name one row; the outputs overlap no input. Deterministic.
 * Errors as in moe_permute. */
MOE_API moe_status moe_unpermute_backward(const void* dy, moe_type dy_type, int64_t dy_stride, const void* rows, moe_type type,
                                          int64_t rows_stride, const int32_t* slot_row, const float* topk_weights,
                                          const moe_dims* d, int64_t H, void* d_rows, int64_t d_rows_stride, float* d_weights,
                                          moe_stream_t stream);

/* ------------------------------------------------------------------------------------------------------
 * 8-bit integers with a scale for each row
 * ------------------------------------------------------------------------------------------------------ */

/* Rows of x in int8 with an fp32 scale each, in the format of MOE_A8W8_INT8's x:
 *   s = max(amax * c, 1e-8), c the fp32 number nearest to 1/127;  q = x / s rounded half to even, within [-127, 127].
 * All fp32, the quotient IEEE's. (moe_dispatch_quantize divides by 127: its s may be one unit in the last place away.)
 * A row that holds a NaN or an infinity gets a NaN or infinite scale and zeros, so products with it are not finite.
 *   x      device [rows, cols] of `type` (bf16 or fp32), x_stride >= cols elements apart
 *   q      device int8 [rows, cols], q_stride >= cols apart;    scale  device fp32 [rows]
 * Errors: MOE_ERR_INVALID_ARG (negative sizes, cols = 0 with rows > 0, cols > 2^30, short strides, a missing pointer, x or
 * scale not aligned to its elements), MOE_ERR_CUDA. */
MOE_API moe_status moe_int8_quantize(const void* x, moe_type type, int64_t rows, int64_t cols, int64_t x_stride, void* q,
                                     int64_t q_stride, float* scale, moe_stream_t stream);

/* out[m,n] = (C[m,n] * b_scale[g,n]) * a_scale[m],  C[m,n] = sum_k a[m,k] * b[g,n,k]
 *   a        int8 [M,K], a_stride apart;                                  a_scale  fp32 [M]
 *   b        int8 [groups][N,K], rows b_stride apart, groups N * b_stride apart;   b_scale  fp32 [groups][N]
 *   offsets  as in moe_fp8_matmul (moe_permute and moe_plan write them)
 *   out      bf16 or fp32 [M,N], out_stride apart
 * C is the exact 32-bit integer, so the result does not depend on the kernel that formed it; it is rounded to fp32, and
 * each product with a scale is. Codes may be -128.
 * Limits: those of moe_fp8_matmul, and K <= 131056 (C stays inside 32 bits). Errors as there. */
typedef struct {
    const void* a;
    const float* a_scale;
    const void* b;
    const float* b_scale;
    const int32_t* offsets;
    void* out;
    int64_t M, N, K;
    int64_t a_stride, b_stride, out_stride;
    int32_t groups;
    int32_t out_type; /* a moe_type */
} moe_int8_matmul_args;

/* Bytes of workspace of moe_int8_matmul for these sizes (0 when they are outside its limits); zeroed once. */
MOE_API size_t moe_int8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t groups);
MOE_API moe_status moe_int8_matmul(const moe_int8_matmul_args* args, void* workspace, size_t workspace_bytes,
                                   moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
