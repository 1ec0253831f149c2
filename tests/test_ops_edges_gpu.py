"""Sizes and values at the edges of the operators of include/moe_ops.h, on the GPU. Bounds are those at the head of
test_ops_gpu.py; where the definition fixes the result (ids, codes, bit patterns), equality is asked for."""
import pytest
import torch

from test_ops_gpu import gen, layer_reference, layer_weights, randn, run_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


# T, H, I, E, K, S: sizes at which whole stages a part would leave the last parts of K without one
@pytest.mark.parametrize("fmt,shape", [("bf16", (1, 3584, 2560, 8, 8, 0)), ("bf16", (1, 2048, 1920, 8, 8, 0)), ("bf16", (2, 128, 4224, 1, 1, 0)),
                                       ("fp8_block", (1, 4096, 6400, 2, 2, 0)), ("fp8_block", (9, 256, 8448, 2, 1, 1)),
                                       ("fp4_mx", (1, 1024, 15360, 2, 2, 0))])
def test_layer_whose_stages_do_not_divide_into_the_parts(moe, fmt, shape):
    T, H, I, E, K, S = shape  # noqa: E741
    g = gen(sum(shape))
    d = moe.dims(*shape)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, fmt))
    ids, weights = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    y, status = run_layer(moe, x, router, w1, w2, d, fmt, ws, topk_ids=ids, topk_weights=weights)
    assert status == moe.MOE_OK
    ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, S)
    assert ((y.double() - ref).abs() <= bound).all(), ((y.double() - ref).abs() / bound).max()
    for _ in range(40):
        again, status = run_layer(moe, x, router, w1, w2, d, fmt, ws)
        assert status == moe.MOE_OK and torch.equal(y, again)


@pytest.mark.parametrize("fmt", ["bf16", "fp8_block", "fp4_mx"])
@pytest.mark.parametrize("T", [3, 12])
def test_layer_that_gives_up_returns(moe, fmt, T):
    """A grid barrier that never fills (its counter starts far below zero) runs into the wait's limit: the launch ends with
    MOE_ERR_TIMEOUT, and the workspace serves again once it is zeroed."""
    H, I, E, K, S = 512, 384, 8, 2, 1  # noqa: E741
    g = gen(21)
    d = moe.dims(T, H, I, E, K, S)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
    want, status = run_layer(moe, x, router, w1, w2, d, fmt)
    assert status == moe.MOE_OK
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(d, fmt))
    ws[:256].view(torch.int32)[1] = -(1 << 24)  # CTAs at the barrier
    _, status = run_layer(moe, x, router, w1, w2, d, fmt, ws)
    assert status == moe.MOE_ERR_TIMEOUT
    moe.moe_ops_workspace_init(ws)
    y, status = run_layer(moe, x, router, w1, w2, d, fmt, ws)
    assert status == moe.MOE_OK and torch.equal(y, want)


def gate_by_definition(rows, K, groups, kept, top):
    """ids from choice values (exact in 32 bits, sums of two as well; -inf and NaN: masked), the groups ranked by what is not masked
    in them."""
    ids = []
    for row in rows:
        on = [v == v and v != float("-inf") for v in row]
        n = len(row) // groups
        rank = []
        for i in range(groups):
            there = sorted(v for v, o in zip(row[i * n:(i + 1) * n], on[i * n:(i + 1) * n]) if o)
            rank.append((bool(there), sum(there[-top:])))
        stay = sorted(range(groups), key=lambda i: (-rank[i][0], -rank[i][1], i))[:kept]
        got = sorted((i for i, o in enumerate(on) if o and i // n in stay), key=lambda i: (-row[i], i))[:K]
        ids.append(got + [-1] * (K - len(got)))
    return ids


def gate_ids(moe, logits, K, **opt):
    T, E = logits.shape
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.moe_gate(logits, moe.dims(T, 128, 128, E, K), ids, w, options=moe.gate_options(**opt))
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_ranks_a_group_by_the_experts_it_has(moe, score):
    inf = float("inf")
    # group 0 masked, one expert left in group 1
    logits = torch.full((1, 8), -inf, device="cuda")
    logits[0, 6] = -2.0
    ids, w = gate_ids(moe, logits, 2, score=score, groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[6, -1]] and w[0, 0] == 1.0 and w[0, 1] == 0.0
    # a NaN masks as -inf does; the sum of one counts against the sum of two (softmax ranks by the logits, sigmoid by scores above 0)
    logits = torch.tensor([[float("nan"), 4.0, -inf, -inf, 1.0, 2.0, -inf, float("nan")]], device="cuda")
    ids, _ = gate_ids(moe, logits, 2, score=score, groups=4, topk_groups=1, group_top=2)
    assert ids.tolist() == ([[1, -1]] if score == "softmax" else [[5, 4]])
    # +inf alone is the highest rank, also beside a masked one
    logits = torch.tensor([[3.0, 3.0, -inf, -inf, -inf, inf, 1.0, 1.0]], device="cuda")
    if score == "softmax":
        ids, _ = gate_ids(moe, logits, 2, score=score, groups=4, topk_groups=1, group_top=2)
        assert ids.tolist() == [[5, -1]]


@pytest.mark.parametrize("groups,kept,top", [(2, 1, 2), (4, 1, 2), (8, 4, 2), (8, 3, 1), (3, 2, 2), (32, 8, 2), (16, 16, 2)])
@pytest.mark.parametrize("left", [0.02, 0.1, 0.5])
def test_gate_groups_with_random_masks(moe, groups, kept, top, left):
    g = gen(groups + kept)
    E, K, T = groups * 8, 5, 60
    logits = torch.randint(-64, 64, (T, E), generator=g, device="cuda") / 8.0
    logits[torch.rand((T, E), generator=g, device="cuda") > left] = float("-inf")
    logits[:, 3] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, float("nan"), logits[:, 3])
    ids, w = gate_ids(moe, logits, K, groups=groups, topk_groups=kept, group_top=top)
    assert ids.tolist() == gate_by_definition(logits.tolist(), K, groups, kept, top)
    assert ((ids < 0) == (w == 0)).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [128, 200, 512])
def test_quantize_keeps_the_sign_of_a_zero(moe, cols, dtype, pow2):
    g = gen(cols)
    x = randn(g, 9, cols)
    x[:, ::3] = -0.0
    x[:, 1::3] = 0.0
    x[1] = -0.0                 # a block of zeros alone: scale 1
    x[2] *= 1e25                # scales outside the range of the exact quotient's short way
    x[3] *= 1e-25
    x[4, 2] = 1e30              # the rest of the block far below a code's smallest value, either sign
    x = x.to(dtype)
    q, scale = torch.empty((9, cols), dtype=torch.uint8, device="cuda"), torch.empty((9, -(-cols // 128)), device="cuda")
    moe.moe_fp8_quantize(x, q, scale, pow2=pow2)
    # the host divides by each scale (IEEE), so -0 and quotients that round to nothing keep their sign
    v = x.float().cpu() / scale.cpu().repeat_interleave(128, 1)[:, :cols]
    assert torch.equal(q.cpu(), v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8))
    assert (q[:, ::3][x[:, ::3] == 0] == 0x80).all() and (scale[1] == 1.0).all()


@pytest.mark.parametrize("apart", [8, 20, 25, 30, 36])
@pytest.mark.parametrize("T,empty", [(2, True), (20, True), (2, False)])
def test_layer_fp4_scales_far_apart(moe, T, empty, apart):
    """One block of 32 in every four has a scale 2^apart times its neighbours'; with `empty` all its codes are zero, so that the
    neighbours alone make the result."""
    H, I, E, K = 512, 256, 4, 2  # noqa: E741
    g = gen(apart)
    d = moe.dims(T, H, I, E, K)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.double, device="cuda")
    table = torch.cat([table, -table])

    def operand(n, k):
        codes = torch.randint(0, 256, (E, n, k // 32, 16), dtype=torch.uint8, generator=g, device="cuda")
        scale = torch.full((E, n, k // 32), 120, dtype=torch.uint8, device="cuda")
        far = torch.randint(0, 4, (E, n, k // 128), generator=g, device="cuda") + 4 * torch.arange(k // 128, device="cuda")
        scale.scatter_(2, far, 120 + apart)
        if empty:
            codes[scale > 120] = 0
        codes = codes.view(E, n, k // 2)
        dense = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
        return codes, scale, dense * torch.exp2(scale.double() - 127).repeat_interleave(32, 2)

    x = randn(g, T, H).to(torch.bfloat16)
    w1, w2 = operand(2 * I, H), operand(H, I)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, K), generator=g, device="cuda")
    y, status = run_layer(moe, x, None, w1, w2, d, "fp4_mx", topk_ids=ids, topk_weights=weights)
    ref, bound = layer_reference(x, ids, weights, w1[2], w2[2], E, 0)
    assert status == moe.MOE_OK
    assert ((y.double() - ref).abs() <= bound).all(), ((y.double() - ref).abs() / bound).max()


def test_layer_workspace_of_the_most_tokens_serves_fewer(moe):
    """14 tokens of these sizes take more memory than 15 (their second product's K is cut into more parts)."""
    T, H, I, E, K = 15, 1024, 8192, 16, 1  # noqa: E741
    g = gen(31)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, "fp8_block", E, 2 * I, H), layer_weights(g, "fp8_block", E, H, I)
    ws = moe.alloc_ops_workspace(moe.moe_layer_workspace_bytes(moe.dims(T, H, I, E, K), "fp8_block"))
    for t in (15, 14, 1, 9):
        d = moe.dims(t, H, I, E, K)
        ids, weights = torch.empty((t, K), dtype=torch.int32, device="cuda"), torch.empty((t, K), device="cuda")
        y, status = run_layer(moe, x[:t], router, w1, w2, d, "fp8_block", ws, topk_ids=ids, topk_weights=weights)
        assert status == moe.MOE_OK
        ref, bound = layer_reference(x[:t], ids, weights, w1[2], w2[2], E, 0)
        assert ((y.double() - ref).abs() <= bound).all()
