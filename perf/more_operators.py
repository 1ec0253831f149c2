"""What the row operators of the MoE path (rows sorted by expert and back, with gradients) and the INT8 product with scales for each
token and channel are measured on.

Every case is a plain dict; `prepare` makes its inputs on the GPU from the seed, `run` makes one pass (the library's calls where
`own` is true, elementary torch operations in 32 bits otherwise), `exact` states the same result in 64 bits.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------


def listed():
    return [
        # a decode step on 8-bit activations: the codes and scales of a handful of tokens go to their experts' rows
        {"name": "permute decode", "op": "permute", "T": 7, "H": 7168, "E": 256, "K": 8, "dtype": "int8", "masked": False},
        # a prefill or training step in bf16, fine-grained experts
        {"name": "permute prefill", "op": "permute", "T": 8192, "H": 7168, "E": 256, "K": 8, "dtype": "bfloat16", "masked": False},
        # the experts' fp32 rows of a decode step back to their tokens, weighted
        {"name": "unpermute decode", "op": "unpermute", "T": 7, "H": 7168, "E": 256, "K": 8, "dtype": "float32", "out": "bfloat16",
         "weighted": True, "masked": False},
        # the same of a prefill step in bf16
        {"name": "unpermute prefill", "op": "unpermute", "T": 8192, "H": 7168, "E": 256, "K": 8, "dtype": "bfloat16", "out": "bfloat16",
         "weighted": True, "masked": False},
        # gradients of the weighted sum: a small fp32 step of odd sizes with masked routes (dropped tokens)
        {"name": "unpermute gradient odd", "op": "unpermute_backward", "T": 333, "H": 1531, "E": 60, "K": 6, "dtype": "float32",
         "out": "float32", "weighted": True, "masked": True},
        # gradients in a training step of a coarse bf16 model
        {"name": "unpermute gradient", "op": "unpermute_backward", "T": 16384, "H": 4096, "E": 8, "K": 2, "dtype": "bfloat16",
         "out": "bfloat16", "weighted": True, "masked": False},
        # activations of a decode step before an INT8 product
        {"name": "quantize decode", "op": "int8_quantize", "M": 3, "K": 7168, "dtype": "bfloat16"},
        # activations of a prefill step
        {"name": "quantize prefill", "op": "int8_quantize", "M": 8192, "K": 7168, "dtype": "bfloat16"},
        # a dense INT8 projection for one token
        {"name": "matmul one row", "op": "int8_matmul", "M": 1, "N": 4096, "K": 7168, "out": "bfloat16", "groups": 1},
        # a batch of decode tokens, an output width that is no multiple of a tile
        {"name": "matmul decode batch", "op": "int8_matmul", "M": 133, "N": 2112, "K": 7168, "out": "float32", "groups": 1},
        # routed rows of a prefill step times their experts' weights, skewed group sizes with empty groups
        {"name": "matmul experts", "op": "int8_matmul", "M": 4099, "N": 4096, "K": 2048, "out": "bfloat16", "groups": 32},
        # a dense INT8 projection of a prefill step
        {"name": "matmul prefill", "op": "int8_matmul", "M": 8192, "N": 4096, "K": 7168, "out": "bfloat16", "groups": 1},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("permute", "unpermute", "unpermute_backward", "int8_quantize", "int8_matmul", "int8_matmul", "int8_matmul"))
    if op == "int8_quantize":
        return {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 100, 7168), "dtype": rng.choice(("bfloat16", "float32"))}
    if op == "int8_matmul":
        groups = rng.choice((1, 1, 1, 8, 32))
        M = _log_int(rng, 1 if groups == 1 else 2 * groups, 8192 if groups == 1 else 4096)
        return {"op": op, "M": M, "N": _log_int(rng, 96, 4096), "K": _log_int(rng, 256, 7168, 16),
                "out": rng.choice(("bfloat16", "float32")), "groups": groups}
    E = rng.randint(4, 256)
    T, H, K = _log_int(rng, 1, 8192), _log_int(rng, 64, 7168), rng.randint(1, min(8, E))
    c = {"op": op, "T": T, "H": H, "E": E, "K": K}
    if op == "permute":
        return {**c, "dtype": rng.choice(("bfloat16", "bfloat16", "float32", "int8")) if T < 4096 else "bfloat16",
                "masked": rng.random() < 0.3}
    return {**c, "dtype": rng.choice(("bfloat16", "float32")) if T < 4096 else "bfloat16", "out": rng.choice(("bfloat16", "float32")),
            "weighted": rng.random() < 0.8, "masked": rng.random() < 0.3}


_SIZE = {"int8": 1, "bfloat16": 2, "float32": 4}


def work(case):
    c = case
    if c["op"] == "int8_quantize":
        return {"bytes": c["M"] * (c["K"] * (_SIZE[c["dtype"]] + 1) + 4), "flops": 3 * c["M"] * c["K"]}
    if c["op"] == "int8_matmul":
        M, N, K, G = c["M"], c["N"], c["K"], c["groups"]
        return {"bytes": M * K + 4 * M + min(G, M) * (N * K + 4 * N) + _SIZE[c["out"]] * M * N, "flops": 2 * M * N * K}
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    one = _SIZE[c["dtype"]]
    if c["op"] == "permute":
        scale = 4 if c["dtype"] == "int8" else 0
        return {"bytes": T * (H * one + scale) * (1 + K) + 12 * T * K + 4 * (E + 1), "flops": T * K}
    tokens, slots = T * H * _SIZE[c["out"]], T * K * H * one
    if c["op"] == "unpermute":
        return {"bytes": tokens + slots + T * K * (4 + 4 * c["weighted"]), "flops": 2 * T * K * H}
    return {"bytes": tokens + 2 * slots + T * K * (8 + 4 * c["weighted"]), "flops": 3 * T * K * H}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _codes(g, *shape):
    """int8 codes and a scale for each row, of normal values whose rows differ in size."""
    x = torch.randn(shape, generator=g, device="cuda") * _randn(g, *shape[:-1], 1).exp()
    scale = (x.abs().amax(-1, keepdim=True) / 127.0).clamp_min(1e-8)
    return torch.round(x / scale).to(torch.int8), scale[..., 0].contiguous()


def _routes(g, c):
    """Expert ids [T,K], distinct in a row, from scores with popular and unpopular experts; masked: one route in ten is -1."""
    popular = _randn(g, c["E"], scale=0.5)
    ids = torch.topk(_randn(g, c["T"], c["E"]) + popular, c["K"], dim=1).indices.to(torch.int32)
    if c["masked"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < 0.1, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _sorted(ids, experts):
    """What sorting by expert gives: row ranges of the experts, the slot of every row (-1 behind the last), the row of every slot."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = (key[None, :] == torch.arange(experts, device=ids.device)[:, None]).sum(1).cumsum(0)
    there = torch.arange(len(flat), device=ids.device) < offsets[-1]
    row_src = torch.where(there, order, torch.full_like(order, -1)).to(torch.int32)
    row = torch.empty_like(order)
    row[order] = torch.arange(len(flat), device=ids.device)
    slot_row = torch.where(flat < 0, torch.full_like(row, -1), row).to(torch.int32).view(ids.shape)
    return offsets, row_src, slot_row


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
    if c["op"] == "int8_quantize":
        rows = _randn(g, c["M"], 1).exp()  # rows of different size, as hidden states have
        s["x"] = (_randn(g, c["M"], c["K"]) * rows).to(getattr(torch, c["dtype"]))
        s["q"] = torch.empty((c["M"], c["K"]), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(c["M"], device="cuda")
    elif c["op"] == "int8_matmul":
        s["a"], s["a_scale"] = _codes(g, c["M"], c["K"])
        s["b"], s["b_scale"] = _codes(g, c["groups"], c["N"], c["K"])
        s["b_scale"] *= c["K"] ** -0.5
        s["out"] = torch.empty((c["M"], c["N"]), dtype=getattr(torch, c["out"]), device="cuda")
        s["offsets"], s["most"] = _group_offsets(g, c["M"], c["groups"]) if c["groups"] > 1 else (None, c["M"])
    else:
        T, H, E, K = c["T"], c["H"], c["E"], c["K"]
        s["ids"], dtype = _routes(g, c), getattr(torch, c["dtype"])
        if c["op"] == "permute":
            s["x"], s["scale"] = _codes(g, T, H) if c["dtype"] == "int8" else (_randn(g, T, H, dtype=dtype), None)
            s["rows"] = torch.zeros((T * K, H), dtype=dtype, device="cuda")
            s["row_scale"] = torch.zeros((T * K, 1), device="cuda")
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["row_src"] = torch.empty(T * K, dtype=torch.int32, device="cuda")
            s["slot_row"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
            if s["scale"] is not None:
                s["scale"] = s["scale"][:, None]
        else:
            s["slot_row"] = _sorted(s["ids"], E)[2]
            s["weights"] = torch.softmax(_randn(g, T, K), -1) if c["weighted"] else None
            s["rows"] = _randn(g, T * K, H, dtype=dtype)
            if c["op"] == "unpermute":
                s["y"] = torch.empty((T, H), dtype=getattr(torch, c["out"]), device="cuda")
            else:
                s["dy"] = _randn(g, T, H, dtype=getattr(torch, c["out"]))
                s["d_rows"] = torch.zeros((T * K, H), dtype=dtype, device="cuda")
                s["d_weights"] = torch.empty((T, K), device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a user's program keeps from call to call: sizes and a workspace."""
    import moe_expert_ffn_topk_gb300 as moe
    c = s["case"]
    if c["op"] == "permute":
        s["d"] = moe.dims(c["T"], 128, 128, c["E"], c["K"])
        s["workspace"] = moe.alloc_ops_workspace(moe.moe_permute_workspace_bytes(s["d"]), "cuda")
    if c["op"] == "int8_matmul":
        s["workspace"] = moe.alloc_ops_workspace(moe.moe_int8_matmul_workspace_bytes(c["M"], c["N"], c["K"], c["groups"]), "cuda")


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_permute(s):
    import moe_expert_ffn_topk_gb300 as moe
    codes = s["scale"] is not None
    moe.moe_permute(s["x"], s["ids"], s["d"], s["rows"], s["offsets"], s["row_src"], s["slot_row"], s["workspace"], scale=s["scale"],
                    row_scale=s["row_scale"] if codes else None)
    out = {"rows": s["rows"], "offsets": s["offsets"], "row_src": s["row_src"], "slot_row": s["slot_row"]}
    return {**out, "row_scale": s["row_scale"]} if codes else out


def _own_unpermute(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_unpermute(s["rows"], s["slot_row"], s["y"], weights=s["weights"])
    return s["y"]


def _own_unpermute_backward(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_unpermute_backward(s["dy"], s["slot_row"], s["d_rows"], weights=s["weights"], rows=s["rows"], d_weights=s["d_weights"])
    return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}


def _own_quantize(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_int8_quantize(s["x"], s["q"], s["scale"])
    return {"q": s["q"], "scale": s["scale"]}


def _own_matmul(s):
    import moe_expert_ffn_topk_gb300 as moe
    moe.moe_int8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], s["workspace"], offsets=s["offsets"])
    return s["out"]


_own = {"permute": _own_permute, "unpermute": _own_unpermute, "unpermute_backward": _own_unpermute_backward,
        "int8_quantize": _own_quantize, "int8_matmul": _own_matmul}


def _plain_permute(s):
    c, ids = s["case"], s["ids"]
    offsets, row_src, slot_row = _sorted(ids, c["E"])
    there = (row_src >= 0)[:, None]
    token = torch.div(row_src.clamp_min(0), c["K"], rounding_mode="floor").long()
    out = {"rows": torch.where(there, s["x"][token], torch.zeros_like(s["rows"])), "offsets": offsets, "row_src": row_src,
           "slot_row": slot_row}
    if s["scale"] is not None:
        out["row_scale"] = torch.where(there, s["scale"][token], torch.zeros_like(s["row_scale"]))
    return out


def _factors(s):
    """The weight of every slot, 0 where the route is masked, in 32 bits [T,K,1]."""
    on = (s["slot_row"] >= 0).float()
    return (on if s["weights"] is None else s["weights"] * on)[..., None]


def _plain_unpermute(s):
    rows = s["rows"][s["slot_row"].clamp_min(0).long()].float()
    return (rows * _factors(s)).sum(1).to(s["y"].dtype)


def _plain_unpermute_backward(s):
    slot, on = s["slot_row"].clamp_min(0).long(), s["slot_row"] >= 0
    dy = s["dy"].float()[:, None, :]
    d_weights = (s["rows"][slot].float() * dy).sum(-1) * on
    d_rows = torch.zeros_like(s["d_rows"])
    d_rows[slot[on]] = (_factors(s) * dy).to(d_rows.dtype)[on]
    return {"d_rows": d_rows, "d_weights": d_weights}


def _plain_quantize(s):
    x = s["x"].float()
    scale = (x.abs().amax(-1) / 127.0).clamp_min(1e-8)
    return {"q": torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8), "scale": scale}


def _plain_matmul(s):
    (m, k), n = s["a"].shape, s["b"].shape[1]
    a, b = s["a"].float(), s["b"].float()
    if s["offsets"] is None:
        return (a @ b[0].T * s["b_scale"] * s["a_scale"][:, None]).to(s["out"].dtype)
    row = torch.arange(m, device=a.device)
    group = (row[:, None] >= s["offsets"][None, 1:]).sum(1)
    place = row - s["offsets"][group]
    full = a.new_zeros((b.shape[0], s["most"], k))
    full[group, place] = a
    product = torch.bmm(full, b.transpose(1, 2))[group, place]
    return (product * s["b_scale"][group] * s["a_scale"][:, None]).to(s["out"].dtype)


_plain = {"permute": _plain_permute, "unpermute": _plain_unpermute, "unpermute_backward": _plain_unpermute_backward,
          "int8_quantize": _plain_quantize, "int8_matmul": _plain_matmul}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "permute":
        rows, row_scale, end = torch.zeros(s["rows"].shape, dtype=torch.double, device="cuda"), s["row_scale"].double(), 0
        for e in range(c["E"]):
            token = (s["ids"] == e).nonzero()[:, 0]  # slot after slot
            rows[end:end + len(token)] = s["x"][token].double() if c["dtype"] != "int8" else 0
            if c["dtype"] == "int8":
                row_scale[end:end + len(token)] = s["scale"].double()[token]
            end += len(token)
        out = {"rows": rows if c["dtype"] != "int8" else None, "offsets": None, "row_src": None, "slot_row": None}
        return {**out, "row_scale": row_scale} if c["dtype"] == "int8" else out
    if c["op"] == "int8_quantize":
        top = s["x"].double().abs().max(1).values
        return {"q": None, "scale": torch.maximum(top / 127, torch.full_like(top, 1e-8))}
    if c["op"] == "int8_matmul":
        out = torch.zeros((c["M"], c["N"]), dtype=torch.double, device="cuda")
        ends = [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()
        for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                product = s["a"][lo:hi].double() @ s["b"][i].double().T
                out[lo:hi] = s["a_scale"][lo:hi].double()[:, None] * product * s["b_scale"][i].double()
        return out
    rows = s["rows"].double()
    y = torch.zeros((c["T"], c["H"]), dtype=torch.double, device="cuda")
    d_rows, d_weights = None, None
    if c["op"] == "unpermute_backward":
        y = s["dy"].double()
        d_rows = torch.zeros_like(rows)
        d_weights = torch.zeros((c["T"], c["K"]), dtype=torch.double, device="cuda")
    for k in range(c["K"]):
        on = (s["slot_row"][:, k] >= 0).nonzero()[:, 0]
        at = s["slot_row"][on, k].long()
        w = torch.ones(len(on), dtype=torch.double, device="cuda") if s["weights"] is None else s["weights"][on, k].double()
        if d_rows is None:
            y[on] += w[:, None] * rows[at]
        else:
            d_rows[at] = w[:, None] * y[on]
            d_weights[on, k] = torch.einsum("th,th->t", rows[at], y[on])
    return y if d_rows is None else {"d_rows": d_rows, "d_weights": d_weights}
