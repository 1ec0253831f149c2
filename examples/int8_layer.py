"""One MoE layer on INT8 weights by its parts, and the routing's gradients.

    python examples/int8_layer.py [tokens]

`by_parts` quantises the tokens once (moe_int8_quantize), sorts their codes and scales by expert (moe_permute), multiplies each expert's rows
by its weights (moe_int8_matmul, grouped), applies SwiGLU, quantises and multiplies again, and adds every token's rows up with its
gate weights (moe_unpermute). `whole` is the same layer in one call (moe_forward, mode a8w8_int8); the program prints how far they
are apart. `gradients` runs the backward pass of a layer whose experts are plain matrices: moe_unpermute_backward for the experts'
outputs and the gate weights, and moe_unpermute without weights for the tokens.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_ffn_topk_gb300 as moe  # noqa: E402


def quantized(x):
    """int8 codes of the rows of x (any leading dimensions) and a scale for each."""
    flat = x.reshape(-1, x.shape[-1])
    q, scale = torch.empty(flat.shape, dtype=torch.int8, device=x.device), torch.empty(len(flat), device=x.device)
    moe.moe_int8_quantize(flat, q, scale)
    return q.view(x.shape), scale.view(x.shape[:-1])


class Layer:
    """Expert weights in int8 with a scale for each output, as moe_forward's mode a8w8_int8 has them."""

    def __init__(self, hidden, inter, experts, topk, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hidden, self.inter, self.experts, self.topk = hidden, inter, experts, topk
        self.router = torch.randn((experts, hidden), generator=g, device="cuda") * hidden ** -0.5
        self.w1, self.s1 = quantized(torch.randn((experts, 2 * inter, hidden), generator=g, device="cuda") * hidden ** -0.5)
        self.w2, self.s2 = quantized(torch.randn((experts, hidden, inter), generator=g, device="cuda") * inter ** -0.5)

    def dims(self, tokens):
        return moe.dims(tokens, self.hidden, self.inter, self.experts, self.topk)

    def routes(self, x):
        ids = torch.empty((len(x), self.topk), dtype=torch.int32, device=x.device)
        weights = torch.empty((len(x), self.topk), device=x.device)
        moe.moe_gate(x.float() @ self.router.T, self.dims(len(x)), ids, weights)
        return ids, weights


def sorted_rows(x, ids, experts, scale=None):
    """Rows of x in the order of their experts, the experts' row ranges, the row of every slot, and the rows' scales."""
    tokens, topk = ids.shape
    d = moe.dims(tokens, 0, 0, experts, topk)
    i32 = dict(dtype=torch.int32, device=x.device)
    rows = torch.empty((tokens * topk, x.shape[1]), dtype=x.dtype, device=x.device)
    offsets, row_src, slot_row = torch.empty(experts + 1, **i32), torch.empty(tokens * topk, **i32), torch.empty((tokens, topk), **i32)
    row_scale = None if scale is None else torch.empty((tokens * topk, 1), device=x.device)
    workspace = moe.alloc_ops_workspace(moe.moe_permute_workspace_bytes(d))  # kept from call to call by a server
    moe.moe_permute(x, ids, d, rows, offsets, row_src, slot_row, workspace, scale=None if scale is None else scale[:, None],
                    row_scale=row_scale)
    return rows, offsets, slot_row, None if scale is None else row_scale[:, 0]


def product(codes, scale, w, w_scale, offsets, dtype):
    out = torch.empty((len(codes), w.shape[1]), dtype=dtype, device=codes.device)
    workspace = moe.alloc_ops_workspace(moe.moe_int8_matmul_workspace_bytes(len(codes), w.shape[1], w.shape[2], w.shape[0]))
    moe.moe_int8_matmul(codes, scale, w, w_scale, out, workspace, offsets=offsets)
    return out


def by_parts(layer, x, ids, weights):
    codes, scale = quantized(x)
    rows, offsets, slot_row, row_scale = sorted_rows(codes, ids, layer.experts, scale)
    h = product(rows, row_scale, layer.w1, layer.s1, offsets, torch.float32)  # (rows without a route hold whatever was there; no slot names what is made of them below)
    act = torch.nn.functional.silu(h[:, :layer.inter]) * h[:, layer.inter:]
    out = product(*quantized(act), layer.w2, layer.s2, offsets, torch.bfloat16)
    y = torch.empty_like(x)
    moe.moe_unpermute(out, slot_row, y, weights=weights)
    return y


def whole(layer, x, ids, weights):
    d = layer.dims(len(x))
    y = torch.empty_like(x)
    moe.moe_forward(*quantized(x), ids, weights, layer.w1, layer.s1, layer.w2, layer.s2, y, d, "a8w8_int8",
                    moe.alloc_workspace(d, "a8w8_int8"))
    return y


def compare(layer, tokens):
    """Relative 2-norm of the difference of the two ways over `tokens` tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((tokens, layer.hidden), generator=g, device="cuda").to(torch.bfloat16)
    ids, weights = layer.routes(x)
    a, b = by_parts(layer, x, ids, weights).float(), whole(layer, x, ids, weights).float()
    return ((a - b).norm() / b.norm()).item()


def gradients(x, ids, weights, experts, dy):
    """y[i] = sum over k of weights[i,k] * (x[i] @ experts[ids[i,k]]) for fp32 x [T,H] and experts [E,H,H]; from dy, the gradients of x, of the
    weights and of the experts."""
    E = len(experts)
    rows, offsets, slot_row, _ = sorted_rows(x, ids, E)
    ends = offsets.tolist()
    out, d_rows, dx, y = (torch.zeros_like(t) for t in (rows, rows, x, x))
    for e in range(E):
        at = slice(ends[e], ends[e + 1])
        out[at] = rows[at] @ experts[e]
    moe.moe_unpermute(out, slot_row, y, weights=weights)
    d_out, d_weights, d_experts = torch.zeros_like(rows), torch.empty_like(weights), torch.empty_like(experts)
    moe.moe_unpermute_backward(dy, slot_row, d_out, weights=weights, rows=out, d_weights=d_weights)
    for e in range(E):
        at = slice(ends[e], ends[e + 1])
        d_rows[at] = d_out[at] @ experts[e].T
        d_experts[e] = rows[at].T @ d_out[at]
    moe.moe_unpermute(d_rows, slot_row, dx)
    return y, dx, d_weights, d_experts


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    print(f"{n} tokens: the two ways are {compare(Layer(1024, 512, 32, 4), n):.4f} apart (relative 2-norm)")
