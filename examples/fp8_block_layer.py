"""One MoE layer on FP8 block-scaled weights, both ways a server runs it:

  - a decode step of a few tokens: moe_layer, everything in one launch;
  - a prefill step of many: moe_gate, moe_plan, then the routed rows in plan order through moe_fp8_quantize and the grouped
    moe_fp8_matmul, twice, with SwiGLU between them.

    python examples/fp8_block_layer.py [tokens]

runs both on the same tokens (as many as moe_layer takes at a time) and prints how far they are apart; the prefill way rounds its
activations to FP8, the decode way does not.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_ffn_topk_gb300 as moe  # noqa: E402

BLOCK = 128


class Layer:
    """Router, expert weights (e4m3 and an fp32 scale for each 128 x 128 block) and gate options of one layer."""

    def __init__(self, hidden, inter, experts, topk, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hidden, self.inter, self.experts, self.topk = hidden, inter, experts, topk
        self.router = (torch.randn((experts, hidden), generator=g, device="cuda") * hidden ** -0.5).to(torch.bfloat16)
        self.bias = 0.05 * torch.randn(experts, generator=g, device="cuda")
        self.options = moe.gate_options(score="sigmoid", groups=4, topk_groups=2, group_top=2, route_scale=2.5)
        self.w1, self.s1 = self._weights(g, 2 * inter, hidden)
        self.w2, self.s2 = self._weights(g, hidden, inter)

    def _weights(self, g, n, k):
        w = torch.randn((self.experts, n // BLOCK, BLOCK, k // BLOCK, BLOCK), generator=g, device="cuda") * k ** -0.5
        scale = w.abs().amax(dim=(2, 4)) / 448.0
        codes = (w / scale[:, :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return codes.view(self.experts, n, k), scale

    def dims(self, tokens):
        return moe.dims(tokens, self.hidden, self.inter, self.experts, self.topk)


def decode(layer, x):
    d = layer.dims(x.shape[0])
    workspace = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, "fp8_block"))  # kept from call to call by a server
    y = torch.empty_like(x)
    moe.moe_layer(x, layer.router, layer.w1, layer.s1, layer.w2, layer.s2, y, d, "fp8_block", workspace, options=layer.options,
                  bias=layer.bias)
    return y


def _product(rows, weights, scales, offsets):
    """Rows in plan order times their experts' weights."""
    m, k = rows.shape
    q = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=rows.device)
    s = torch.empty((m, -(-k // BLOCK)), device=rows.device)
    moe.moe_fp8_quantize(rows, q, s)
    groups, n = weights.shape[:2]
    out = torch.empty((m, n), dtype=torch.bfloat16, device=rows.device)
    workspace = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(m, n, k, groups))
    moe.moe_fp8_matmul(q, s, weights, scales, out, workspace, offsets=offsets)
    return out


def prefill(layer, x):
    tokens, d = x.shape[0], layer.dims(x.shape[0])
    ids = torch.empty((tokens, layer.topk), dtype=torch.int32, device=x.device)
    weights = torch.empty((tokens, layer.topk), device=x.device)
    moe.moe_gate(x.float() @ layer.router.float().T, d, ids, weights, bias=layer.bias, options=layer.options)
    counts = torch.empty(layer.experts, dtype=torch.int32, device=x.device)
    offsets = torch.empty(layer.experts + 1, dtype=torch.int32, device=x.device)
    row_src = torch.empty(tokens * layer.topk, dtype=torch.int32, device=x.device)
    moe.moe_plan(ids, d, moe.alloc_workspace(d, "a16w16"), counts, offsets, row_src)
    token = (row_src // layer.topk).long()
    h = _product(x[token], layer.w1, layer.s1, offsets).float()
    act = (torch.nn.functional.silu(h[:, :layer.inter]) * h[:, layer.inter:]).to(torch.bfloat16)
    rows = _product(act, layer.w2, layer.s2, offsets).float() * weights.view(-1)[row_src.long(), None]
    return torch.zeros((tokens, layer.hidden), device=x.device).index_add_(0, token, rows).to(torch.bfloat16)


def compare(layer, tokens):
    """Relative 2-norm of the two ways' difference over `tokens` tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((tokens, layer.hidden), generator=g, device="cuda").to(torch.bfloat16)
    many = prefill(layer, x).float()
    step = moe.MOE_LAYER_MAX_TOKENS
    few = torch.cat([decode(layer, x[i:i + step].contiguous()) for i in range(0, tokens, step)]).float()
    return ((many - few).norm() / few.norm()).item()


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    print(f"{n} tokens: the two ways are {compare(Layer(1024, 512, 32, 4), n):.4f} apart (relative 2-norm)")
