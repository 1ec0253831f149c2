"""What the router, the block-scaled FP8 product and the few-token MoE layer are measured on.

Every case is a plain dict; `prepare` makes its inputs on the GPU from the seed, `run` makes one pass (the library's calls where
`own` is true, elementary torch operations in 32 bits otherwise), `exact` states the same result in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128          # columns (and weight rows) that share one FP8 scale
E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------


def listed():
    return [
        # the router of a decode step: a handful of tokens, sigmoid scores with a selection bias, experts in groups
        {"name": "gate decode", "op": "gate", "T": 7, "E": 256, "K": 8, "score": "sigmoid", "groups": 8, "topk_groups": 4,
         "bias": True, "dtype": "float32"},
        # the router of a prefill step, softmax scores, logits straight from a bf16 product (ties happen)
        {"name": "gate prefill", "op": "gate", "T": 8192, "E": 60, "K": 4, "score": "softmax", "groups": 1, "topk_groups": 1,
         "bias": False, "dtype": "bfloat16"},
        # activations of one decode step before an FP8 product
        {"name": "quantize decode", "op": "quantize", "M": 3, "K": 7168, "dtype": "bfloat16", "pow2": False},
        # activations of a prefill step, power-of-two scales
        {"name": "quantize prefill", "op": "quantize", "M": 8192, "K": 7168, "dtype": "bfloat16", "pow2": True},
        # a dense FP8 projection for one token
        {"name": "matmul one row", "op": "matmul", "M": 1, "N": 4096, "K": 7168, "out": "bfloat16", "groups": 1},
        # a batch of decode tokens, an output width that ends inside a block of 128
        {"name": "matmul decode batch", "op": "matmul", "M": 133, "N": 2112, "K": 7168, "out": "float32", "groups": 1},
        # a dense FP8 projection of a prefill step
        {"name": "matmul prefill", "op": "matmul", "M": 8192, "N": 4096, "K": 7168, "out": "bfloat16", "groups": 1},
        # routed rows of a prefill step times their experts' weights, skewed group sizes with empty groups
        {"name": "matmul experts", "op": "matmul", "M": 4099, "N": 4096, "K": 2048, "out": "bfloat16", "groups": 32},
        # the layer of a fine-grained model for one user: top-8 of 256 and a shared expert, FP8 block weights
        {"name": "layer fp8 one token", "op": "layer", "T": 1, "H": 7168, "I": 2048, "E": 256, "K": 8, "S": 1,
         "weights": "fp8_block", "score": "sigmoid", "groups": 8, "topk_groups": 4, "bias": True},
        # the layer of a coarse bf16 model for a few users
        {"name": "layer bf16 few tokens", "op": "layer", "T": 3, "H": 4096, "I": 14336, "E": 8, "K": 2, "S": 0,
         "weights": "bf16", "score": "softmax", "groups": 1, "topk_groups": 1, "bias": False},
        # a small fine-grained layer on FP4 weights, where latency counts
        {"name": "layer fp4 small", "op": "layer", "T": 5, "H": 2048, "I": 768, "E": 64, "K": 6, "S": 0,
         "weights": "fp4_mx", "score": "softmax", "groups": 1, "topk_groups": 1, "bias": False},
        # a decode batch that touches most of the 256 experts
        {"name": "layer fp8 decode batch", "op": "layer", "T": 32, "H": 7168, "I": 2048, "E": 256, "K": 8, "S": 1,
         "weights": "fp8_block", "score": "sigmoid", "groups": 8, "topk_groups": 4, "bias": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    n = min(hi, max(lo, int(round(v / step)) * step))
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(("gate", "quantize", "matmul", "matmul", "layer", "layer"))
    if op == "gate":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * rng.randint(4, 256 // groups)
        score = rng.choice(("softmax", "sigmoid"))
        kept = max(1, groups // 2)
        return {"op": op, "T": _log_int(rng, 1, 8192), "E": E, "K": rng.randint(1, min(8, kept * (E // groups))), "score": score,
                "groups": groups, "topk_groups": kept, "bias": score == "sigmoid" and rng.random() < 0.7,
                "dtype": rng.choice(("float32", "bfloat16"))}
    if op == "quantize":
        return {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 128, 7168, 8),
                "dtype": rng.choice(("bfloat16", "float32")), "pow2": rng.random() < 0.5}
    if op == "matmul":
        groups = rng.choice((1, 1, 1, 8, 32))
        N, K = _log_int(rng, 96, 4096), _log_int(rng, 256, 7168, 16)
        M = _log_int(rng, 1 if groups == 1 else 4 * groups, 8192 if groups == 1 else 4096)
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(("bfloat16", "float32")), "groups": groups}
    weights = rng.choice(("fp8_block", "fp8_block", "bf16", "fp4_mx"))
    H, I = 128 * rng.choice([n for n in range(4, 33) if n != 24]), 128 * _log_int(rng, 3, 23)  # noqa: E741
    E = rng.choice((8, 16, 60, 64, 128))
    if E <= 16:
        I = 2 * I + 128  # noqa: E741
    score = rng.choice(("softmax", "sigmoid"))
    groups = 4 if E % 4 == 0 and rng.random() < 0.4 else 1
    return {"op": op, "T": _log_int(rng, 1, 32), "H": H, "I": I, "E": E, "K": rng.randint(2, 2 if E <= 16 else 8),
            "S": rng.choice((0, 0, 1)), "weights": weights, "score": score, "groups": groups,
            "topk_groups": 2 if groups == 4 else 1, "bias": score == "sigmoid"}


def _parts(n, block=BLOCK):
    return -(-n // block)


def work(case):
    c = case
    if c["op"] == "gate":
        size = 2 if c["dtype"] == "bfloat16" else 4
        return {"bytes": c["T"] * (c["E"] * size + 8 * c["K"]) + 4 * c["E"] * bool(c["bias"]), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "quantize":
        size = 2 if c["dtype"] == "bfloat16" else 4
        return {"bytes": c["M"] * (c["K"] * (size + 1) + 4 * _parts(c["K"])), "flops": 2 * c["M"] * c["K"]}
    if c["op"] == "matmul":
        M, N, K, G = c["M"], c["N"], c["K"], c["groups"]
        out = 2 if c["out"] == "bfloat16" else 4
        used = min(G, M)
        return {"bytes": M * K + 4 * M * _parts(K) + used * (N * K + 4 * _parts(N) * _parts(K)) + out * M * N,
                "flops": 2 * M * N * K}
    T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "S"))  # noqa: E741
    # experts that T independent draws of K of E touch, on average
    touched = E * (1.0 - (1.0 - K / E) ** T) + S
    per = {"bf16": 2.0, "fp8_block": 1.0 + 4.0 / BLOCK ** 2, "fp4_mx": 0.5 + 1.0 / 32}[c["weights"]]
    return {"bytes": int(touched * 3 * H * I * per + 2 * E * H + 4 * T * H),
            "flops": 6 * T * (K + S) * H * I + 2 * T * E * H}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _fp8_weight(g, n, k):
    """One weight [n, k]: normal values, e4m3 codes, an fp32 scale for each 128 x 128 block (the last ones may be smaller)."""
    w = torch.randn((n, k), generator=g, device="cuda")
    nb, kb = _parts(n), _parts(k)
    full = torch.zeros((nb * BLOCK, kb * BLOCK), device="cuda")
    full[:n, :k] = w * k ** -0.5
    full = full.view(nb, BLOCK, kb, BLOCK)
    scale = full.abs().amax(dim=(1, 3)).clamp_min(1e-12) / E4M3_MAX
    q = (full / scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _fp8_weights(g, groups, n, k):
    codes = torch.empty((groups, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((groups, _parts(n), _parts(k)), device="cuda")
    for i in range(groups):
        codes[i], scales[i] = _fp8_weight(g, n, k)
    return codes, scales


def _fp4_weights(g, groups, n, k):
    """e2m1 codes, two in a byte (the even element in the low nibble), a power-of-two scale byte for each 32 of k."""
    codes = torch.empty((groups, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((groups, n, k // 32), dtype=torch.uint8, device="cuda")
    for i in range(groups):
        w = torch.randn((n, k // 32, 32), generator=g, device="cuda") * k ** -0.5
        e = torch.ceil(torch.log2(w.abs().amax(-1).clamp_min(1e-12) / 6.0))
        a = (w * torch.exp2(-e)[..., None]).view(n, k)
        steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        c = torch.bucketize(a.abs(), steps).to(torch.uint8) | ((a < 0).to(torch.uint8) << 3)
        codes[i] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[i] = (e + 127.0).to(torch.uint8)
    return codes, scales


def _quantize(x):
    """Rows of x in e4m3 with an fp32 scale for each 128 columns."""
    m, k = x.shape
    kb = _parts(k)
    full = torch.zeros((m, kb * BLOCK), device=x.device)
    full[:, :k] = x
    full = full.view(m, kb, BLOCK)
    scale = full.abs().amax(-1).clamp_min(1e-12) / E4M3_MAX
    q = (full / scale[..., None]).view(m, kb * BLOCK)[:, :k]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).contiguous(), scale


def _group_offsets(g, rows, groups):
    """Row ranges of `groups` groups: sizes from a skewed popularity, a few of them empty."""
    p = 1.0 / torch.arange(1, groups + 1, device="cuda") ** 0.7
    p = p[torch.randperm(groups, generator=g, device="cuda")]
    p[:: max(4, groups // 4)] = 0.0
    pick = torch.multinomial(p, rows, replacement=True, generator=g)
    counts = torch.bincount(pick, minlength=groups)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def prepare(case, seed):
    g, c = _generator(seed), case
    s = {"case": c}
    if c["op"] == "gate":
        s["logits"] = _randn(g, c["T"], c["E"], dtype=getattr(torch, c["dtype"]))
        s["bias"] = _randn(g, c["E"], scale=0.05) if c["bias"] else None
        s["ids"] = torch.empty((c["T"], c["K"]), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((c["T"], c["K"]), device="cuda")
    elif c["op"] == "quantize":
        rows = _randn(g, c["M"], 1).exp()  # rows of different size, as hidden states have
        s["x"] = (_randn(g, c["M"], c["K"]) * rows).to(getattr(torch, c["dtype"]))
        s["q"] = torch.empty((c["M"], c["K"]), dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty((c["M"], _parts(c["K"])), device="cuda")
    elif c["op"] == "matmul":
        s["a"], s["a_scale"] = _quantize(_randn(g, c["M"], c["K"]) * _randn(g, c["M"], 1).exp())
        s["b"], s["b_scale"] = _fp8_weights(g, c["groups"], c["N"], c["K"])
        s["out"] = torch.empty((c["M"], c["N"]), dtype=getattr(torch, c["out"]), device="cuda")
        s["offsets"], s["most"] = _group_offsets(g, c["M"], c["groups"]) if c["groups"] > 1 else (None, c["M"])
    else:
        T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "S"))  # noqa: E741
        s["x"] = _randn(g, T, H, dtype=torch.bfloat16)
        s["router"] = _randn(g, E, H, scale=H ** -0.5, dtype=torch.bfloat16)
        s["bias"] = _randn(g, E, scale=0.05) if c["bias"] else None
        if c["weights"] == "bf16":  # [experts, in, out]
            s["w1"] = torch.empty((E + S, H, 2 * I), dtype=torch.bfloat16, device="cuda")
            s["w2"] = torch.empty((E + S, I, H), dtype=torch.bfloat16, device="cuda")
            for w in (s["w1"], s["w2"]):
                for i in range(E + S):
                    w[i] = torch.randn(w.shape[1:], generator=g, device="cuda") * w.shape[1] ** -0.5
            s["w1_scale"] = s["w2_scale"] = None
        else:  # [experts, out, in]
            make = _fp8_weights if c["weights"] == "fp8_block" else _fp4_weights
            s["w1"], s["w1_scale"] = make(g, E + S, 2 * I, H)
            s["w2"], s["w2_scale"] = make(g, E + S, H, I)
        s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    if c["op"] in ("gate", "layer"):
        s["route_scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a user's program keeps from call to call: sizes, options and a workspace."""
    import moe_expert_ffn_topk_gb300 as moe
    c = s["case"]
    if c["op"] in ("gate", "layer"):
        s["d"] = moe.dims(c["T"], c.get("H", 128), c.get("I", 128), c["E"], c["K"], c.get("S", 0))
        s["options"] = moe.gate_options(score=c["score"], groups=c["groups"], topk_groups=c["topk_groups"], group_top=2,
                                        normalize=True, route_scale=s["route_scale"])
    if c["op"] == "matmul":
        s["workspace"] = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(c["M"], c["N"], c["K"], c["groups"]), "cuda")
    if c["op"] == "layer":
        s["workspace"] = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(s["d"], c["weights"]), "cuda")


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_gate(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_gate(s["logits"], s["d"], s["ids"], s["weights"], bias=s["bias"], options=s["options"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _own_quantize(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_fp8_quantize(s["x"], s["q"], s["scale"], pow2=s["case"]["pow2"])
    return {"q": s["q"], "scale": s["scale"]}


def _own_matmul(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], s["workspace"], offsets=s["offsets"])
    return s["out"]


def _own_layer(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_layer(s["x"], s["router"], s["w1"], s["w1_scale"], s["w2"], s["w2_scale"], s["y"], s["d"], s["case"]["weights"],
                  s["workspace"], options=s["options"], bias=s["bias"])
    return s["y"]


_own = {"gate": _own_gate, "quantize": _own_quantize, "matmul": _own_matmul, "layer": _own_layer}


def _top(values, k):
    """The k largest of each row, largest first, ties to the lowest index."""
    order = torch.sort(values, dim=-1, descending=True, stable=True).indices
    return order[..., :k]


def _route(logits, c, bias, route_scale):
    x = logits.float()
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score + bias if bias is not None else x if c["score"] == "softmax" else score
    T, E = x.shape
    if c["groups"] > 1:
        grouped = choice.view(T, c["groups"], -1)
        best = torch.sort(grouped, dim=-1, descending=True).values[..., :2].sum(-1)
        kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=x.device)
        kept.scatter_(1, _top(best, c["topk_groups"]), True)
        choice = torch.where(kept[..., None], grouped, torch.full_like(grouped, -math.inf)).view(T, E)
    ids = _top(choice, c["K"])
    w = torch.gather(score, 1, ids)
    w = w / (w.sum(-1, keepdim=True) + 1e-20) * route_scale
    return ids.to(torch.int32), w


def _plain_gate(s):
    ids, w = _route(s["logits"], s["case"], s["bias"], s["route_scale"])
    return {"ids": ids, "weights": w}


def _plain_quantize(s):
    x = s["x"].float()
    m, k = x.shape
    pad = _parts(k) * BLOCK - k
    if pad:
        x = torch.cat([x, x.new_zeros((m, pad))], 1)
    x = x.view(m, -1, BLOCK)
    scale = x.abs().amax(-1) / E4M3_MAX
    if s["case"]["pow2"]:
        # the next power of two: any fraction bit carries into the exponent
        scale = ((scale.view(torch.int32) + 0x7FFFFF) & -0x800000).view(torch.float32)
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(m, -1)[:, :k].to(torch.float8_e4m3fn)
    return {"q": q, "scale": scale}


def _spread(scale, n, k):
    """A scale for each element from one for each block of 128 x 128."""
    return scale.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _plain_matmul(s):
    (m, k), n = s["a"].shape, s["b"].shape[1]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    b = s["b"].float() * _spread(s["b_scale"], n, k)
    if s["offsets"] is None:
        return (a @ b[0].T).to(s["out"].dtype)
    row = torch.arange(m, device=a.device)
    group = (row[:, None] >= s["offsets"][None, 1:]).sum(1)
    place = row - s["offsets"][group]
    full = a.new_zeros((b.shape[0], s["most"], k))
    full[group, place] = a
    return torch.bmm(full, b.transpose(1, 2))[group, place].to(s["out"].dtype)


def _expert_weights(s, ids):
    """w1 [slots, 2I, H] and w2 [slots, H, I] of the experts `ids`, in 32 bits."""
    c, out = s["case"], []
    for name in ("w1", "w2"):
        w = s[name].view(torch.uint8 if c["weights"] == "fp8_block" else s[name].dtype)[ids]
        if c["weights"] == "bf16":
            out.append(w.float().transpose(1, 2))
        elif c["weights"] == "fp8_block":
            w = w.view(torch.float8_e4m3fn)
            nb, kb = s[name + "_scale"].shape[1:]
            scale = s[name + "_scale"][ids]
            out.append((w.float().view(-1, nb, BLOCK, kb, BLOCK) * scale[:, :, None, :, None]).view(w.shape))
        else:
            table = torch.tensor(E2M1, device=w.device)
            v = torch.stack([table[(w & 15).int()], table[(w >> 4).int()]], -1).view(*w.shape[:2], -1, 32)
            scale = torch.exp2(s[name + "_scale"][ids].float() - 127.0)
            out.append((v * scale[..., None]).view(w.shape[0], w.shape[1], -1))
    return out


def _swiglu(h, inter):
    gate, up = h[..., :inter], h[..., inter:]
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_layer(s):
    c = s["case"]
    T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "S"))  # noqa: E741
    x = s["x"].float()
    ids, w = _route(x @ s["router"].float().T, c, s["bias"], s["route_scale"])
    w1, w2 = _expert_weights(s, ids.flatten().long())
    a = _swiglu(torch.bmm(w1, x.repeat_interleave(K, 0)[..., None])[..., 0], I)
    del w1
    slots = torch.bmm(w2, a[..., None])[..., 0].view(T, K, H)
    del w2
    y = (slots * w[..., None]).sum(1)
    if S:
        w1, w2 = _expert_weights(s, torch.arange(E, E + S, device=x.device))
        a = _swiglu(torch.einsum("th,enh->ten", x, w1), I)
        y = y + torch.einsum("tei,ehi->th", a, w2)
    return y.to(torch.bfloat16)


_plain = {"gate": _plain_gate, "quantize": _plain_quantize, "matmul": _plain_matmul, "layer": _plain_layer}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------


def _route64(logits, c, bias, route_scale):
    """ids and weights of every token, one row at a time on the host for the selection."""
    x = logits.double().cpu()
    s = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    choice = s if bias is None else s + bias.double().cpu()
    if bias is None and c["score"] == "softmax":
        choice = x
    rows, per = choice.numpy(), x.shape[1] // c["groups"]
    ids = []
    for row in rows:
        allowed = range(len(row))
        if c["groups"] > 1:
            best = [sum(sorted(row[i * per:(i + 1) * per])[-2:]) for i in range(c["groups"])]
            kept = sorted(range(c["groups"]), key=lambda i: (-best[i], i))[:c["topk_groups"]]
            allowed = [i for i in allowed if i // per in kept]
        ids.append(sorted(allowed, key=lambda i: (-row[i], i))[:c["K"]])
    ids = torch.tensor(ids, dtype=torch.long)
    w = s.gather(1, ids)
    return ids, w / w.sum(-1, keepdim=True) * route_scale


def _dense64(s, name, e):
    """Expert e's weight as [out, in]."""
    c, w = s["case"], s[name][e]
    if c["weights"] == "bf16":
        return w.double().T
    if c["weights"] == "fp8_block":
        return w.double() * torch.kron(s[name + "_scale"][e].double(), torch.ones((BLOCK, BLOCK), dtype=torch.double, device=w.device))
    n = w.shape[0]
    v = torch.empty((n, 2 * w.shape[1]), dtype=torch.double, device=w.device)
    for half, code in ((0, w & 15), (1, w >> 4)):
        mag, exp = (code & 1).double(), ((code >> 1) & 3).double()
        value = torch.where(exp == 0, 0.5 * mag, (1.0 + 0.5 * mag) * torch.exp2(exp - 1.0))
        v[:, half::2] = torch.where(code >= 8, -value, value)
    return v * torch.exp2(s[name + "_scale"][e].double() - 127.0).repeat_interleave(32, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gate":
        _, w = _route64(s["logits"], c, s["bias"], s["route_scale"])
        return {"ids": None, "weights": w}
    if c["op"] == "quantize":
        x = s["x"].double()
        q, scales = torch.zeros_like(x), []
        for j in range(0, c["K"], BLOCK):
            part = x[:, j:j + BLOCK]
            top = part.abs().max(1).values / E4M3_MAX
            if c["pow2"]:
                mantissa, exponent = torch.frexp(top)
                top = torch.where(top > 0, torch.exp2((exponent - (mantissa == 0.5).int()).double()), top)
            top = torch.where(top > 0, top, torch.ones_like(top))
            v = part / top[:, None]
            ulp = torch.exp2((torch.frexp(v).exponent - 1).clamp_min(-6).double() - 3.0)
            q[:, j:j + BLOCK] = torch.round(v / ulp) * ulp
            scales.append(top)
        return {"q": q, "scale": torch.stack(scales, 1)}
    if c["op"] == "matmul":
        m, n, k = c["M"], c["N"], c["K"]
        out = torch.zeros((m, n), dtype=torch.double, device="cuda")
        ends = [0, m] if s["offsets"] is None else s["offsets"].tolist()
        for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
            for kb in range(_parts(k)):
                cols = slice(kb * BLOCK, min(k, (kb + 1) * BLOCK))
                part = s["a"][lo:hi, cols].double() @ s["b"][i][:, cols].double().T
                scale = s["b_scale"][i, :, kb].double().repeat_interleave(BLOCK)[:n]
                out[lo:hi] += part * s["a_scale"][lo:hi, kb].double()[:, None] * scale
        return out
    x, inter = s["x"].double(), c["I"]
    ids, w = _route64(x @ s["router"].double().T, c, s["bias"], s["route_scale"])
    ids, w = ids.to(x.device), w.to(x.device)
    y = torch.zeros_like(x)
    for e in range(c["E"] + c["S"]):
        weight = (w * (ids == e)).sum(1) if e < c["E"] else torch.ones(c["T"], dtype=torch.double, device=x.device)
        rows = weight.nonzero()[:, 0]
        if len(rows):
            h = x[rows] @ _dense64(s, "w1", e).T
            a = h[:, :inter] * torch.sigmoid(h[:, :inter]) * h[:, inter:]
            y[rows] += weight[rows, None] * (a @ _dense64(s, "w2", e).T)
    return y
