"""The operators of include/moe_ops.h against plain 64-bit implementations on the GPU.

Tolerances, fixed before the first run:
  - gate weights: fp32 exp (2 ulp), sums of at most 1024 terms in a tree (10 + 5 roundings) and two divides: below 40
    roundings of 2^-24, so 2^-18 relative.
  - products: every product of two 8- or 16-bit operands is exact in fp32; a sum over at most 128 of them on the tensor cores
    may drop bits below 2^-22 of the running sum at each of its additions: 128 * 2^-22 = 2^-15 of the sum of magnitudes.
    Adding the blocks in fp32 is far below that. Then the output's own rounding (bf16 has 8 significant bits: 2^-8 to nearest).
  - the layer: the products' bound on gate and up sums, carried through SwiGLU (|SiLU'| < 1.1), one rounding of the
    activations to at least 11 bits (2^-11), and the second product's bound.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

SUM_EPS = 2.0 ** -15
BF16_EPS = 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ---------------------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------------------


def gate_call(moe, logits, K, bias=None, **opt):
    T, E = logits.shape
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    moe.moe_gate(logits, moe.dims(T, 128, 128, E, K), ids, w, bias=bias, options=moe.gate_options(**opt) if opt else None)
    return ids.cpu(), w.cpu()


def gate_reference(logits, K, bias=None, score="softmax", groups=1, topk_groups=1, group_top=1, normalize=True, route_scale=1.0):
    """Row by row in Python: ids by the definition on 64-bit choice values, their weights, and the choice values."""
    ids, weights, choices = [], [], []
    for row in logits.double().cpu().tolist():
        on = [v == v and v != -math.inf for v in row]
        if score == "softmax":
            top = max((v for v, o in zip(row, on) if o), default=0.0)
            e = [(1.0 if v == top else 0.0) if top == math.inf else math.exp(v - top) if o else 0.0 for v, o in zip(row, on)]
            s = [v / max(sum(e), 1e-300) for v in e]
        else:
            s = [(1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0) if o else 0.0 for v, o in zip(row, on)]
        c = [a + b for a, b in zip(s, bias.double().tolist())] if bias is not None else (row if score == "softmax" else s)
        c = [v if o else -math.inf for v, o in zip(c, on)]
        if groups > 1:
            n = len(c) // groups
            rank = [sum(sorted(c[i * n:(i + 1) * n])[-group_top:]) for i in range(groups)]
            kept = sorted(range(groups), key=lambda i: (-rank[i], i))[:topk_groups]
            c = [v if i // n in kept else -math.inf for i, v in enumerate(c)]
        got = [i for i in sorted(range(len(c)), key=lambda i: (-c[i], i)) if c[i] != -math.inf][:K]
        w = [s[i] for i in got]
        total = sum(w) + 1e-20 if normalize else 1.0
        ids.append(got + [-1] * (K - len(got)))
        weights.append([v / total * route_scale for v in w] + [0.0] * (K - len(got)))
        choices.append(c)
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.double), torch.tensor(choices, dtype=torch.double)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (5, 60, 4), (130, 64, 6), (3, 256, 8), (2, 300, 32), (9, 512, 8),
                                   (4, 1000, 10), (7, 33, 32)])
def test_gate_softmax_ids_and_ties(moe, T, E, K, dtype):
    # multiples of 1/8: many equal logits, decided by the index
    logits = (torch.randint(-24, 24, (T, E), generator=gen(E + T), device="cuda") / 8.0).to(dtype)
    ids, w = gate_call(moe, logits, K)
    ref_ids, ref_w, _ = gate_reference(logits, K)
    assert torch.equal(ids, ref_ids)
    torch.testing.assert_close(w.double(), ref_w, rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (8, 4, 2), (8, 3, 1), (4, 2, 2), (32, 8, 2), (2, 1, 2)])
@pytest.mark.parametrize("normalize", [True, False])
def test_gate_sigmoid_groups(moe, groups, kept, top, normalize):
    logits = torch.randint(-32, 32, (37, 256), generator=gen(groups), device="cuda") / 8.0
    opt = dict(score="sigmoid", groups=groups, topk_groups=kept, group_top=top, normalize=normalize, route_scale=2.5)
    ids, w = gate_call(moe, logits, 8, **opt)
    ref_ids, ref_w, _ = gate_reference(logits, 8, **opt)
    if top == 1 or groups == 1:
        # sums of two sigmoids that differ in 64 bits may be equal in 32; single values of this grid are not
        assert torch.equal(ids, ref_ids)
    same = (ids == ref_ids).all(1)
    assert same.float().mean() > 0.9
    torch.testing.assert_close(w.double()[same], ref_w[same], rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("score,groups,kept", [("sigmoid", 8, 4), ("softmax", 1, 1), ("sigmoid", 1, 1), ("softmax", 6, 2)])
def test_gate_bias(moe, score, groups, kept):
    g = gen(3)
    E, K = 240, 8
    logits, bias = randn(g, 65, E), 0.1 * randn(g, E)
    opt = dict(score=score, groups=groups, topk_groups=kept, group_top=2)
    ids, w = gate_call(moe, logits, K, bias=bias, **opt)
    ref_ids, ref_w, choice = gate_reference(logits, K, bias=bias.cpu(), **opt)
    # values of 0..1.5 in fp32: choices that are nearer than 1e-6 may come in either order
    got, want = choice.gather(1, ids.long()), choice.gather(1, ref_ids.long())
    assert (got - want).abs().max() < 1e-6
    same = (ids == ref_ids).all(1)
    assert same.float().mean() > 0.95
    torch.testing.assert_close(w.double()[same], ref_w[same], rtol=2.0 ** -18, atol=0)


def test_gate_masks(moe):
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    rows = [[-inf] * 8, [nan] * 8, [-inf, 1.0] + [-inf] * 6, [nan, 2.0, -inf, 1.0, nan, 3.0, -inf, -inf], [low] * 8,
            [low, 0.0] + [low] * 6, [inf, 1.0, inf] + [0.0] * 5, [0.0, -0.0] * 4, [3e38, 3e38, -3e38, 1.0, 0, 0, 0, 0]]
    logits = torch.tensor(rows, device="cuda")
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            ids, w = gate_call(moe, logits, 4, score=score, normalize=normalize)
            ref_ids, ref_w, _ = gate_reference(logits, 4, score=score, normalize=normalize)
            assert torch.equal(ids, ref_ids), (score, ids, ref_ids)
            torch.testing.assert_close(w.double(), ref_w, rtol=2.0 ** -18, atol=1e-37)
    # a group whose every expert is masked, next to others
    logits = torch.zeros((1, 16), device="cuda")
    logits[0, :12] = -inf
    ids, w = gate_call(moe, logits, 6, groups=4, topk_groups=2, group_top=2)
    assert ids[0].tolist() == [12, 13, 14, 15, -1, -1] and w[0].tolist() == [0.25] * 4 + [0.0, 0.0]


def test_gate_strided_rows_and_stream(moe):
    g = gen(9)
    wide = randn(g, 40, 200)
    logits = wide[::2, 17:81]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids, w = gate_call(moe, logits, 5)
    ref_ids, ref_w, _ = gate_reference(logits, 5)
    assert torch.equal(ids, ref_ids)
    torch.testing.assert_close(w.double(), ref_w, rtol=2.0 ** -18, atol=0)


# ---------------------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------------------


def quantize_reference(x, pow2):
    """fp32 on the host: IEEE divide and round half to even are the definition, so codes and scales are equal bit for bit."""
    x = x.float().cpu()
    m, k = x.shape
    codes, scales = torch.zeros((m, k), dtype=torch.uint8), torch.zeros((m, -(-k // 128)))
    for b in range(scales.shape[1]):
        part = x[:, b * 128:(b + 1) * 128]
        s = part.abs().amax(1) / 448.0
        if pow2:
            s = torch.where(s > 0, torch.exp2(torch.ceil(torch.log2(s.double()))).float(), s)
        s = torch.where(s == 0, torch.ones_like(s), s)
        q = (part / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        codes[:, b * 128:(b + 1) * 128] = q.view(torch.uint8)
        scales[:, b] = s
    return codes, scales


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,pad", [(1, 1, 0), (1, 128, 0), (3, 7168, 0), (130, 512, 0), (5, 200, 0), (7, 1000, 24), (4, 255, 1),
                                     (2, 2112, 5), (1000, 384, 0)])
def test_quantize(moe, m, k, pad, dtype, pow2):
    g = gen(m * 7 + k)
    wide = (randn(g, m, k + pad) * torch.exp(3 * randn(g, m, 1))).to(dtype)
    x = wide[:, :k]
    if m > 2:
        x[1] = 0
    q = torch.full((m, k + pad), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((m, -(-k // 128)), float("nan"), device="cuda")
    moe.moe_fp8_quantize(x, q[:, :k], scale, pow2=pow2)
    codes, scales = quantize_reference(x, pow2)
    assert torch.equal(scale.cpu(), scales)
    assert torch.equal(q[:, :k].cpu(), codes)
    assert (q[:, k:] == 0x55).all()


def test_quantize_extremes(moe):
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    x = torch.zeros((5, 128), device="cuda")
    x[0, 3], x[1, 5], x[2, 7], x[3, 9], x[3, 10], x[4, 1] = big, tiny, math.inf, math.nan, 1.0, -448.0
    q, scale = torch.empty((5, 128), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((5, 1), device="cuda")
    moe.moe_fp8_quantize(x, q, scale)
    v = q.float() * scale
    assert v[0, 3] == torch.tensor(big / 448.0).float() * 448.0 and v[0].count_nonzero() == 1
    assert torch.isfinite(v[1]).all() and scale[1] > 0
    assert not torch.isfinite(v[2, 7]) and torch.isnan(v[3, 9]) and v[4, 1] == -448.0


# ---------------------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------------------


def fp8_operand(g, rows, k, pad=0, block_rows=1):
    codes = (randn(g, rows, k + pad) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.exp(randn(g, -(-rows // block_rows), -(-k // 128))) * 2.0 ** -6
    return codes[:, :k], scale


def matmul_reference(a, a_scale, b, b_scale, offsets):
    """The definition and the sum of magnitudes, in 64 bits; rows that belong to no group are NaN."""
    (m, k), n = a.shape, b.shape[1]
    ends = [0, m] if offsets is None else offsets.tolist()
    out = torch.full((m, n), float("nan"), dtype=torch.double, device="cuda")
    mag = torch.zeros_like(out)
    ad = a.double() * a_scale.double().repeat_interleave(128, 1)[:, :k]
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        bd = b[i].double() * b_scale[i].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        out[lo:hi] = ad[lo:hi] @ bd.T
        mag[lo:hi] = ad[lo:hi].abs() @ bd.abs().T
    return out, mag


def check_matmul(moe, m, n, k, out_dtype, groups=1, sizes=None, pads=(0, 0, 0), seed=0, empty_tail=0):
    g = gen(seed + m + 3 * n + 7 * k)
    a, a_scale = fp8_operand(g, m, k, pads[0])
    parts = [fp8_operand(g, n, k, pads[1], 128) for _ in range(groups)]
    b_wide = torch.zeros((groups, n, k + pads[1]), dtype=torch.uint8, device="cuda")
    for i, (codes, _) in enumerate(parts):
        b_wide[i, :, :k] = codes.view(torch.uint8)
    b = b_wide.view(torch.float8_e4m3fn)[:, :, :k]
    b_scale = torch.stack([s for _, s in parts])
    offsets = None
    if sizes is not None:
        offsets = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32, device="cuda")
    wide = torch.full((m, n + pads[2]), -7.0, dtype=out_dtype, device="cuda")
    out = wide[:, :n]
    ws = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(m, n, k, groups))
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, out, ws, offsets=offsets)
    assert moe.moe_check_device_error(ws) == moe.MOE_OK
    ref, mag = matmul_reference(a, a_scale, b, b_scale, offsets)
    eps = BF16_EPS if out_dtype == torch.bfloat16 else 2.0 ** -23
    done = ~torch.isnan(ref[:, 0])
    err = (out.double() - ref)[done].abs()
    assert torch.isfinite(out[done]).all()
    assert (err <= SUM_EPS * mag[done] + eps * ref[done].abs() + 1e-30).all(), (err / (SUM_EPS * mag[done] + 1e-30)).max()
    assert (out[~done] == -7.0).all() and (wide[:, n:] == -7.0).all()
    first = out.clone()
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, out, ws, offsets=offsets)  # the workspace as the first call left it
    assert torch.equal(first, out)


MATMUL_SIZES = [(1, 1, 16), (1, 128, 128), (1, 4096, 7168), (2, 129, 144), (3, 100, 2048), (7, 2112, 1024), (8, 256, 512),
                (9, 96, 400), (16, 4000, 256), (17, 640, 1040), (31, 128, 384), (33, 257, 272), (64, 512, 2048), (65, 192, 128),
                (100, 1000, 1008), (127, 384, 640), (128, 128, 128), (129, 2112, 896), (200, 130, 7168), (256, 256, 256),
                (300, 4096, 512), (513, 576, 1536), (1000, 1001, 720)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", MATMUL_SIZES)
def test_matmul(moe, m, n, k, out_dtype):
    check_matmul(moe, m, n, k, out_dtype)


@pytest.mark.parametrize("m,n,k", [(2, 64, 80), (5, 200, 256), (40, 333, 208), (140, 300, 384), (260, 512, 1040)])
@pytest.mark.parametrize("pads", [(16, 0, 0), (0, 48, 1), (32, 16, 8)])
def test_matmul_strides(moe, m, n, k, pads):
    check_matmul(moe, m, n, k, torch.bfloat16, pads=pads)
    check_matmul(moe, m, n, k, torch.float32, pads=pads)


@pytest.mark.parametrize("n,k", [(128, 128), (256, 512), (200, 272), (1024, 384)])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 5], [3, 0, 1, 2], [128, 128], [130, 0, 1, 255, 64], [1] * 40, [0] * 7 + [300],
                                   [17, 300, 2, 0, 129, 1, 1, 500]])
def test_matmul_groups(moe, n, k, sizes):
    check_matmul(moe, sum(sizes), n, k, torch.bfloat16, groups=len(sizes), sizes=sizes)
    check_matmul(moe, sum(sizes) + 5, n, k, torch.float32, groups=len(sizes), sizes=sizes)  # rows after the last group


def test_matmul_offsets_out_of_range_are_clamped(moe):
    """Offsets outside [0, M], or decreasing ones, touch no row outside the matrix."""
    g = gen(1)
    m, n, k = 70, 96, 128
    a, a_scale = fp8_operand(g, m, k)
    b, b_scale = fp8_operand(g, 3 * n, k, 0, 96)
    b, b_scale = b.view(3, n, k), b_scale.view(3, 1, 1)
    ws = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(m, n, k, 3))
    guard = torch.full((m + 64, n), -7.0, device="cuda")
    out = guard[32:32 + m]
    for offsets in ([-5, 20, 1000, 1 << 30], [0, 50, 20, 70], [-(1 << 31), -1, 0, 0]):
        out.fill_(-7.0)
        moe.moe_fp8_matmul(a, a_scale, b, b_scale, out, ws, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        assert moe.moe_check_device_error(ws) == moe.MOE_OK
        assert (guard[:32] == -7.0).all() and (guard[32 + m:] == -7.0).all()
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, out, ws, offsets=torch.tensor([-5, 20, 1000, 1 << 30], dtype=torch.int32, device="cuda"))
    ref, mag = matmul_reference(a, a_scale, b, b_scale, torch.tensor([0, 20, 70, 70]))
    assert ((out.double() - ref).abs() <= SUM_EPS * mag + 2.0 ** -23 * ref.abs()).all()


@pytest.mark.parametrize("m", [1, 20, 300])
def test_matmul_nan_stays_in_its_row_and_column(moe, m):
    g = gen(5)
    n, k = 256, 512
    a, a_scale = fp8_operand(g, m, k)
    b, b_scale = fp8_operand(g, n, k, 0, 128)
    a, b = a.contiguous(), b.contiguous()
    b.view(torch.uint8)[77, 300] = 0x7F  # NaN code
    if m > 1:
        a_scale[m // 2, 2] = math.inf
    out = torch.empty((m, n), device="cuda")
    ws = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(m, n, k))
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, out, ws)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[:, 77] = True
    if m > 1:
        want[m // 2] = True
    assert torch.equal(bad, want)


def test_matmul_on_another_stream(moe):
    g = gen(6)
    a, a_scale = fp8_operand(g, 40, 512)
    b, b_scale = fp8_operand(g, 300, 512, 0, 128)
    ws = moe.alloc_ops_workspace(moe.moe_fp8_matmul_workspace_bytes(40, 300, 512))
    here, there = torch.empty((40, 300), device="cuda"), torch.empty((40, 300), device="cuda")
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, here, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_fp8_matmul(a, a_scale, b, b_scale, there, ws, stream=s)
    s.synchronize()
    assert torch.equal(here, there)


# ---------------------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def layer_weights(g, fmt, experts, n, k):
    """Random weights in the format: the tensors of the call and the dense [experts, n, k] values in 64 bits."""
    if fmt == "bf16":
        w = (randn(g, experts, k, n) * k ** -0.5).to(torch.bfloat16)
        return w, None, w.double().transpose(1, 2)
    if fmt == "fp8_block":
        codes = (randn(g, experts, n, k) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.exp(0.5 * randn(g, experts, n // 128, k // 128)) * (0.01 * k ** -0.5)
        dense = codes.double() * scale.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        return codes, scale, dense
    codes = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, generator=g, device="cuda")
    scale = torch.randint(118, 124, (experts, n, k // 32), dtype=torch.uint8, generator=g, device="cuda")
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.double, device="cuda")
    dense = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return codes, scale, dense * torch.exp2(scale.double() - 127).repeat_interleave(32, 2)


def layer_reference(x, ids, weights, w1, w2, E, S, clamp=None):
    """y and its bound (see the head of this file) from the ids and weights that were used, in 64 bits."""
    x = x.double()
    T, H = x.shape
    inter = w2.shape[2]
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E + S):
        gate = ((ids == e) * weights.double()).sum(1) if e < E else torch.ones(T, dtype=torch.double, device="cuda")
        rows = (ids == e).any(1).nonzero()[:, 0] if e < E else torch.arange(T, device="cuda")
        if not len(rows):
            continue
        h, mag = x[rows] @ w1[e].T, x[rows].abs() @ w1[e].abs().T
        a, u = h[:, :inter], h[:, inter:]
        if clamp is not None:
            a, u = a.clamp(-clamp, clamp), u.clamp(-clamp, clamp)
        silu = a * torch.sigmoid(a)
        act = silu * u
        d_act = 2.0 ** -11 * act.abs() + SUM_EPS * (1.1 * mag[:, :inter] * u.abs() + mag[:, inter:] * silu.abs())
        y[rows] += gate[rows, None] * (act @ w2[e].T)
        bound[rows] += gate[rows, None].abs() * ((d_act + SUM_EPS * act.abs()) @ w2[e].abs().T)
    return y, bound + BF16_EPS * y.abs() + 1e-30


LAYER_SHAPES = [(1, 128, 128, 1, 1, 0), (1, 256, 128, 8, 2, 1), (3, 512, 384, 8, 2, 0), (5, 384, 256, 60, 6, 0), (8, 1024, 128, 32, 4, 1),
                (9, 256, 640, 16, 3, 2), (17, 640, 128, 300, 8, 0), (33, 256, 256, 12, 4, 1), (64, 384, 128, 5, 5, 0),
                (64, 128, 256, 3, 1, 0), (40, 896, 384, 128, 8, 1), (1, 7168, 2048, 16, 8, 1), (12, 4224, 1152, 20, 3, 0),
                (64, 2048, 4096, 4, 2, 1)]
FORMATS = ["bf16", "fp8_block", "fp4_mx"]


def run_layer(moe, x, router, w1, w2, d, fmt, ws=None, **kw):
    y = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, fmt))
    moe.moe_layer(x, router, w1[0], w1[1], w2[0], w2[1], y, d, fmt, ws, **kw)
    return y, moe.moe_check_device_error(ws)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", LAYER_SHAPES)
def test_layer(moe, fmt, shape):
    T, H, I, E, K, S = shape  # noqa: E741
    g = gen(sum(shape))
    d = moe.dims(*shape)
    x = randn(g, T, H).to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, fmt))
    for router_dtype in (torch.bfloat16, torch.float32):
        router = (randn(g, E, H) * H ** -0.5).to(router_dtype)
        ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
        weights = torch.full((T, K), float("nan"), device="cuda")
        y, status = run_layer(moe, x, router, w1, w2, d, fmt, ws, topk_ids=ids, topk_weights=weights)
        assert status == moe.MOE_OK
        # the router: logits are sums of H exact products in fp32, below 1e-5 off for sizes of about 1
        logits = x.double() @ router.double().T
        got, want = logits.gather(1, ids.long()), logits.topk(K, 1).values
        assert (got - want).abs().max() < 1e-5
        assert (weights.double() - torch.softmax(got, 1)).abs().max() < 2e-5
        ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, S)
        assert torch.isfinite(y).all()
        assert ((y.double() - ref).abs() <= bound).all(), ((y.double() - ref).abs() / bound).max()
        again, _ = run_layer(moe, x, router, w1, w2, d, fmt, ws)
        assert torch.equal(y, again)


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_sigmoid_groups_bias_clamp(moe, fmt):
    T, H, I, E, K, S = 6, 256, 256, 64, 8, 1  # noqa: E741
    g = gen(11)
    d = moe.dims(T, H, I, E, K, S)
    x, router, bias = (3 * randn(g, T, H)).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5), 0.05 * randn(g, E)
    w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
    opt = moe.gate_options(score="sigmoid", groups=8, topk_groups=4, group_top=2, route_scale=2.5)
    ids, weights = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    y, status = run_layer(moe, x, router, w1, w2, d, fmt, options=opt, bias=bias, topk_ids=ids, topk_weights=weights,
                          activation_clamp=0.75)
    assert status == moe.MOE_OK
    # the same selection as moe_gate's on logits from a 64-bit product
    gate_ids, gate_w = torch.empty_like(ids), torch.empty_like(weights)
    moe.moe_gate((x.double() @ router.double().T).float(), d, gate_ids, gate_w, bias=bias, options=opt)
    assert torch.equal(ids, gate_ids)
    torch.testing.assert_close(weights, gate_w, rtol=1e-5, atol=0)
    ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, S, clamp=0.75)
    assert ((y.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 4, 21, 64])
def test_layer_with_given_routes(moe, fmt, T):
    """Masked routes, rows that route nowhere, many tokens on one expert, repeated experts, experts outside the range."""
    H, I, E, K = 256, 128, 6, 3  # noqa: E741
    g = gen(T)
    d = moe.dims(T, H, I, E, K)
    x = randn(g, T, H).to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E, 2 * I, H), layer_weights(g, fmt, E, H, I)
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, fmt))
    weights = torch.rand((T, K), generator=g, device="cuda") - 0.3
    ids = torch.randint(-1, E, (T, K), dtype=torch.int32, generator=g, device="cuda")
    one = torch.full_like(ids, -1)
    one[:, 1] = 4
    none = torch.full_like(ids, -1)
    twice = ids.clone()
    twice[:, 2] = twice[:, 0]
    for case in (ids, one, none, twice):
        y, status = run_layer(moe, x, None, w1, w2, d, fmt, ws, topk_ids=case, topk_weights=weights)
        assert status == moe.MOE_OK
        dense = torch.zeros((T, E), dtype=torch.double, device="cuda")
        for k in range(K):
            on = case[:, k] >= 0
            dense[on] = dense[on].scatter_add(1, case[on, k:k + 1].long(), weights[on, k:k + 1].double())
        every = torch.where((case[:, :, None] == torch.arange(E, device="cuda")).any(1), torch.arange(E, device="cuda"), -1)
        ref, bound = layer_reference(x, every, dense, w1[2], w2[2], E, 0)
        extra = torch.zeros_like(bound)
        for k in range(K):  # a repeated expert's two products are rounded apart: their magnitudes add
            _, b = layer_reference(x, case[:, k:k + 1], weights[:, k:k + 1], w1[2], w2[2], E, 0)
            extra += b
        assert ((y.double() - ref).abs() <= torch.maximum(bound, extra)).all()
        assert (y[(case < 0).all(1)] == 0).all()
    bad = ids.clone()
    bad[0, 0], bad[-1, 2] = E, -2
    y, status = run_layer(moe, x, None, w1, w2, d, fmt, ws, topk_ids=bad, topk_weights=weights)
    assert status == moe.MOE_ERR_BAD_ROUTE
    good = torch.where((bad < 0) | (bad >= E), -1, bad)
    same, status = run_layer(moe, x, None, w1, w2, d, fmt, ws, topk_ids=good, topk_weights=weights)
    assert status == moe.MOE_OK and torch.equal(y, same)


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_extremes(moe, fmt):
    """Large, tiny and zero rows keep their accuracy; an infinite or NaN row stays alone."""
    T, H, I, E, K = 7, 256, 128, 4, 2  # noqa: E741
    g = gen(2)
    d = moe.dims(T, H, I, E, K)
    x = randn(g, T, H)
    x[1] *= 1e-6
    x[2] *= 1e4
    x[3] = 0
    x = x.to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E, 2 * I, H), layer_weights(g, fmt, E, H, I)
    ids = torch.tensor([[0, 1], [1, 2], [2, 3], [3, 0], [0, 2], [1, 3], [0, 3]], dtype=torch.int32, device="cuda")
    weights = torch.rand((T, K), generator=g, device="cuda")
    y, status = run_layer(moe, x, None, w1, w2, d, fmt, topk_ids=ids, topk_weights=weights)
    ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, 0)
    assert status == moe.MOE_OK and ((y.double() - ref).abs() <= bound).all() and (y[3] == 0).all()
    x[4, 7], x[5, 9] = math.inf, math.nan
    z, _ = run_layer(moe, x, None, w1, w2, d, fmt, topk_ids=ids, topk_weights=weights)
    assert not torch.isfinite(z[4]).any() and torch.isnan(z[5]).all()
    keep = [0, 1, 2, 3, 6]
    assert torch.equal(z[keep], y[keep])


def test_layer_workspace_of_other_sizes(moe):
    """One workspace, zeroed once, serves calls of different sizes and formats in turn."""
    big = moe.dims(64, 512, 512, 32, 4, 1)
    ws = moe.alloc_ops_workspace(max(moe.moe_layer_workspace_bytes(big, f) for f in FORMATS))
    g = gen(8)
    for shape, fmt in (((64, 512, 512, 32, 4, 1), "fp8_block"), ((1, 128, 128, 4, 2), "bf16"), ((30, 512, 256, 8, 2), "fp4_mx"),
                       ((2, 256, 512, 32, 4, 1), "fp8_block"), ((64, 128, 128, 9, 1), "bf16")):
        T, H, I, E, K = shape[:5]  # noqa: E741
        S = shape[5] if len(shape) > 5 else 0
        d = moe.dims(*shape)
        x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
        w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
        shared, status = run_layer(moe, x, router, w1, w2, d, fmt, ws)
        fresh, _ = run_layer(moe, x, router, w1, w2, d, fmt)
        assert status == moe.MOE_OK and torch.equal(shared, fresh)


def test_layer_in_a_graph(moe):
    T, H, I, E, K = 4, 256, 128, 16, 2  # noqa: E741
    g = gen(4)
    d = moe.dims(T, H, I, E, K)
    router = (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, "fp8_block", E, 2 * I, H), layer_weights(g, "fp8_block", E, H, I)
    x, y = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, "fp8_block"))
    call = lambda: moe.moe_layer(x, router, w1[0], w1[1], w2[0], w2[1], y, d, "fp8_block", ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        x.copy_(randn(g, T, H))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        call()
        assert torch.equal(got, y) and y.abs().sum() > 0


# ---------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------


def test_gate_feeds_the_routed_layer(moe):
    """moe_gate's ids and weights in moe_forward give what moe_layer gives, on the same bf16 weights."""
    T, H, I, E, K, S = 24, 256, 256, 8, 2, 1  # noqa: E741
    g = gen(12)
    d = moe.dims(T, H, I, E, K, S)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, "bf16", E + S, 2 * I, H), layer_weights(g, "bf16", E + S, H, I)
    ids, weights = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.moe_gate(x.float() @ router.float().T, d, ids, weights)
    y, ws = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), moe.alloc_workspace(d, "a16w16")
    moe.moe_forward(x, None, ids, weights, w1[0], None, w2[0], None, y, d, "a16w16", ws)
    ours, status = run_layer(moe, x, router, w1, w2, d, "bf16")
    assert status == moe.MOE_OK
    # moe_forward rounds A and every combine row to bf16 (2^-8 each, of terms whose magnitudes the bound sums)
    ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, S)
    assert (y.double() - ref).abs().max() <= 2e-2 * ref.abs().max()
    assert ((ours.double() - ref).abs() <= bound).all()


def test_example_runs_both_ways(moe):
    """The example's decode and prefill ways agree up to the prefill way's FP8 rounding: x and the activations each lose
    2^-4 a value at most, 2^-4/sqrt(3) in the mean of uniform errors: together below 2^-4 * sqrt(2/3) = 0.051."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_block_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_block_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.compare(example.Layer(1024, 512, 32, 4), 150) < 0.051
