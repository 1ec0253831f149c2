"""moe_permute, moe_unpermute and moe_unpermute_backward against plain 64-bit implementations on the GPU.

What moves (rows, scales, whole numbers) has to be equal. Tolerances of what is computed, fixed before the first run, with
u = 2^-24 for a rounding to fp32 and 2^-8 for one to bf16, S the sum of the magnitudes of the terms:
  - y: K fused multiply-adds, K u S, and the rounding to y's type;
  - d_rows: one fp32 product and the rounding to the rows' type;
  - d_weights: H products added in fp32 in some order, (H + 8) u S.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def routes(g, T, E, K, masked=0.0):
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)  # the same expert twice in a token, too
    return torch.where(torch.rand((T, K), generator=g, device="cuda") < masked, torch.full_like(ids, -1), ids)


def sort_by_definition(ids, E):
    flat = ids.flatten().tolist()
    order = sorted((s for s, e in enumerate(flat) if 0 <= e < E), key=lambda s: (flat[s], s))
    row = [-1] * len(flat)
    for p, s in enumerate(order):
        row[s] = p
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + flat.count(e) if len(flat) < 5000 else 0)
    if len(flat) >= 5000:
        offsets = [0] + torch.bincount(torch.tensor([flat[s] for s in order] or [0]), minlength=E)[:E].mul(bool(order)).cumsum(0).tolist()
    return offsets, order + [-1] * (len(flat) - len(order)), row


def permute(moe, x, ids, E, scale=None, rows=None, **kw):
    T, K = ids.shape
    d = moe.dims(T, 0, 0, E, K)
    if rows is None:
        rows = torch.full((T * K, x.shape[1]), 7, device="cuda").to(x.dtype)
    out = dict(offsets=torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
               row_src=torch.full((T * K,), -7, dtype=torch.int32, device="cuda"),
               slot_row=torch.full((T, K), -7, dtype=torch.int32, device="cuda"))
    row_scale = None if scale is None else torch.full((T * K, scale.shape[1]), 7.0, device="cuda")
    ws = moe.alloc_ops_workspace(moe.moe_permute_workspace_bytes(d))
    moe.moe_permute(x, ids, d, rows, out["offsets"], out["row_src"], out["slot_row"], ws, scale=scale, row_scale=row_scale, **kw)
    return rows, out, row_scale, moe.moe_check_device_error(ws)


def values(g, T, H, dtype):
    if dtype in (torch.int8, torch.uint8):
        return torch.randint(0, 127, (T, H), generator=g, device="cuda").to(dtype)
    x = torch.randn((T, H), generator=g, device="cuda")
    return x.to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8)


# the last sizes sort in launches of their own (more than 4096 slots, or many tokens of a slot each), runs of slots that end inside a group of 32
SIZES = [(1, 1, 1, 1), (1, 64, 4, 4), (3, 100, 5, 2), (7, 7168, 256, 8), (64, 384, 1024, 32), (65, 130, 3, 1), (341, 33, 60, 6),
         (342, 33, 60, 6), (683, 64, 1, 3), (2049, 24, 1000, 1), (1111, 520, 64, 7), (4096, 16, 256, 8), (9000, 8, 7, 3), (4096, 40, 5, 1),
         (4097, 40, 5, 1), (5001, 24, 1000, 1), (1366, 33, 1024, 3),
         (512, 72, 256, 8), (2048, 16, 64, 1), (2049, 16, 64, 1), (4096, 16, 1, 1), (1449, 8, 6, 2)]


@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("T,H,E,K", SIZES)
def test_permute_is_a_stable_sort(moe, T, H, E, K, masked):
    g = gen(T + H)
    ids = routes(g, T, E, K, masked)
    x = values(g, T, H, torch.bfloat16)
    rows, out, _, status = permute(moe, x, ids, E)
    assert status == moe.MOE_OK
    offsets, row_src, slot_row = sort_by_definition(ids, E)
    assert out["offsets"].tolist() == offsets and out["row_src"].tolist() == row_src
    assert out["slot_row"].flatten().tolist() == slot_row
    R = offsets[-1]
    token = torch.tensor(row_src[:R], dtype=torch.long, device="cuda") // K
    assert torch.equal(bits(rows[:R]), bits(x[token]))
    assert (rows[R:] == 7).all()  # rows behind the last are left alone


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int8, torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("T,H", [(9, 48), (9, 51), (700, 33), (700, 64)])
def test_permute_types_and_scales(moe, dtype, T, H):
    g = gen(H)
    x = values(g, T, H, dtype)
    ids = routes(g, T, 16, 4, 0.1)
    scale = torch.randn((T, 3), generator=g, device="cuda")
    rows, out, row_scale, status = permute(moe, x, ids, 16, scale=scale)
    R = int(out["offsets"][-1])
    token = out["row_src"][:R].long() // 4
    assert status == moe.MOE_OK and torch.equal(bits(rows[:R]), bits(x)[token])
    assert torch.equal(row_scale[:R], scale[token]) and (row_scale[R:] == 7).all()


@pytest.mark.parametrize("T", [5, 1000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int8])
@pytest.mark.parametrize("start,H", [(0, 40), (8, 40), (1, 40), (3, 37), (2, 36), (4, 44)])
def test_permute_strided_rows(moe, T, dtype, start, H):
    """Columns [start, start + H) of wider matrices: every alignment of a row's start."""
    g = gen(start)
    wide = values(g, T, 64, dtype)
    ids = routes(g, T, 8, 3, 0.2)
    out_wide = torch.full((T * 3, 80), 9, device="cuda").to(dtype)
    rows, out, _, status = permute(moe, wide[:, start:start + H], ids, 8, rows=out_wide[:, start:start + H])
    R = int(out["offsets"][-1])
    assert status == moe.MOE_OK and torch.equal(rows[:R], wide[out["row_src"][:R].long() // 3, start:start + H])
    assert (out_wide[:, :start] == 9).all() and (out_wide[:, start + H:] == 9).all() and (out_wide[R:] == 9).all()


@pytest.mark.parametrize("T", [6, 3000])
def test_permute_reports_bad_ids(moe, T):
    g = gen(1)
    ids = routes(g, T, 4, 2)
    ids[1, 0], ids[2, 1], ids[4, 1] = 4, -2, 2 ** 31 - 1
    x = values(g, T, 32, torch.float32)
    rows, out, _, status = permute(moe, x, ids, 4)
    assert status == moe.MOE_ERR_BAD_ROUTE
    offsets, row_src, slot_row = sort_by_definition(ids, 4)
    assert out["offsets"].tolist() == offsets and out["row_src"].tolist() == row_src and out["slot_row"].flatten().tolist() == slot_row
    R = offsets[-1]
    assert R == 2 * T - 3 and torch.equal(rows[:R], x[out["row_src"][:R].long() // 2])


def test_permute_empty_and_all_masked(moe):
    rows, out, _, status = permute(moe, torch.zeros((0, 8), device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert status == moe.MOE_OK and out["offsets"].tolist() == [0] * 6
    for T in (4, 2000):
        ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
        rows, out, _, status = permute(moe, torch.ones((T, 8), device="cuda"), ids, 5)
        assert status == moe.MOE_OK and out["offsets"].tolist() == [0] * 6
        assert (out["row_src"] == -1).all() and (out["slot_row"] == -1).all() and (rows == 7).all()


def unpermute_reference(rows, slot_row, weights):
    T, K = slot_row.shape
    y, size = (torch.zeros((T, rows.shape[1]), dtype=torch.double, device="cuda") for _ in range(2))
    for k in range(K):
        on = (slot_row[:, k] >= 0).nonzero()[:, 0]
        r = rows[slot_row[on, k].long()].double()
        w = 1.0 if weights is None else weights[on, k].double()[:, None]
        y[on] += w * r
        size[on] += (w * r).abs()
    return y, size


def slots(g, T, K, masked):
    """slot_row of a permutation, some slots without a row."""
    row = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32).view(T, K)
    return torch.where(torch.rand((T, K), generator=g, device="cuda") < masked, torch.full_like(row, -1), row).contiguous()


BACK = [(1, 1, 1), (1, 8, 1), (2, 7168, 8), (5, 129, 6), (33, 1000, 32), (300, 40, 9), (1500, 264, 4), (800, 2051, 8), (60, 2048, 2),
        (400, 4096, 7), (4099, 1032, 2), (1000, 517, 1), (2500, 1000, 3), (950, 517, 4), (4801, 248, 7),
        (3001, 504, 5), (9800, 63, 3), (5000, 121, 3), (60, 1532, 6), (700, 132, 5)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,K", BACK)
def test_unpermute(moe, T, H, K, dtype, out, weighted):
    g = gen(T * K + H)
    rows, slot_row = torch.randn((T * K, H), generator=g, device="cuda").to(dtype), slots(g, T, K, 0.2)
    w = torch.randn((T, K), generator=g, device="cuda") if weighted else None
    slot_row[0] = -1  # a token without any route
    y = torch.full((T, H), float("nan"), device="cuda").to(out)
    moe.moe_unpermute(rows, slot_row, y, weights=w)
    ref, size = unpermute_reference(rows, slot_row, w)
    sum_error = K * U * size
    assert ((y.double() - ref).abs() <= sum_error + HALF_STEP[out] * (ref.abs() + sum_error)).all()
    assert (y[0] == 0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,K", BACK)
def test_unpermute_backward(moe, T, H, K, dtype, out, weighted):
    g = gen(T * K + H)
    rows, slot_row = torch.randn((T * K, H), generator=g, device="cuda").to(dtype), slots(g, T, K, 0.2)
    dy = torch.randn((T, H), generator=g, device="cuda").to(out)
    w = torch.randn((T, K), generator=g, device="cuda") if weighted else None
    d_rows, d_w = torch.full_like(rows, 9), torch.full((T, K), float("nan"), device="cuda")
    moe.moe_unpermute_backward(dy, slot_row, d_rows, weights=w, rows=rows, d_weights=d_w)
    on = slot_row >= 0
    named = torch.zeros(T * K, dtype=torch.bool, device="cuda")
    named[slot_row[on].long()] = True
    assert (d_rows[~named] == 9).all() and (d_w[~on] == 0).all()
    token = torch.arange(T, device="cuda")[:, None].expand(T, K)[on]
    factor = torch.ones(len(token), device="cuda") if w is None else w[on]
    ref = dy[token].double() * factor.double()[:, None]
    got = d_rows[slot_row[on].long()].double()
    product = 0.0 if w is None else U
    assert ((got - ref).abs() <= ref.abs() * (product + HALF_STEP[dtype] * (1 + product))).all()
    terms = dy[token].double() * rows[slot_row[on].long()].double()
    assert ((d_w[on].double() - terms.sum(1)).abs() <= (H + 8) * U * terms.abs().sum(1)).all()
    # without the weights' gradient: the same d_rows, rows not needed
    again = torch.full_like(rows, 9)
    moe.moe_unpermute_backward(dy, slot_row, again, weights=w)
    assert torch.equal(again, d_rows)


def test_gradients_against_differences(moe):
    """The sum of y's products with dy changes with the weights and the rows as the gradients say (the function is linear in each, so a
    difference over a power of two is exact but for y's rounding)."""
    g = gen(4)
    T, H, K = 6, 72, 3
    rows, slot_row = torch.randn((T * K, H), generator=g, device="cuda"), slots(g, T, K, 0.2)
    w, dy = torch.randn((T, K), generator=g, device="cuda"), torch.randn((T, H), generator=g, device="cuda")
    d_rows, d_w = torch.zeros_like(rows), torch.empty_like(w)
    moe.moe_unpermute_backward(dy, slot_row, d_rows, weights=w, rows=rows, d_weights=d_w)

    def loss(rows, w):
        y = torch.empty((T, H), device="cuda")
        moe.moe_unpermute(rows, slot_row, y, weights=w)
        return (y.double() * dy.double()).sum(), 4 * K * U * (unpermute_reference(rows, slot_row, w)[1] * dy.double().abs()).sum()
    base, off = loss(rows, w)
    for at in [(0, 0), (2, 1), (5, 2)]:
        more = w.clone()
        more[at] += 0.5
        step = (more[at].double() - w[at].double())
        value, off2 = loss(rows, more)
        assert abs((value - base) / step - d_w[at].double()) <= (off + off2) / step + (H + 8) * U * 100
    for at in [(0, 0), (7, 70), (17, 3)]:
        more = rows.clone()
        more[at] += 0.5
        step = (more[at].double() - rows[at].double())
        value, off2 = loss(more, w)
        assert abs((value - base) / step - d_rows[at].double()) <= (off + off2) / step + 1e-5


def test_unpermute_masks_what_it_does_not_read(moe):
    """NaN and infinite weights of masked slots and rows that no slot names change nothing; entries outside the rows are masked."""
    g = gen(2)
    T, H, K = 5, 64, 4
    rows, slot_row = torch.randn((T * K, H), generator=g, device="cuda"), slots(g, T, K, 0.0)
    w = torch.randn((T, K), generator=g, device="cuda")
    clean = slot_row.clone()
    clean[1, 2], clean[3, 0] = -1, -1
    slot_row[1, 2], slot_row[3, 0] = T * K, -(2 ** 31)
    bad_rows, bad_w = rows.clone(), w.clone()
    bad_w[1, 2], bad_w[3, 0] = float("nan"), math.inf
    named = torch.zeros(T * K, dtype=torch.bool, device="cuda")
    named[clean[clean >= 0].long()] = True
    bad_rows[~named] = float("nan")
    a, b = torch.empty((T, H), device="cuda"), torch.empty((T, H), device="cuda")
    moe.moe_unpermute(rows, clean, a, weights=w)
    moe.moe_unpermute(bad_rows, slot_row, b, weights=bad_w)
    assert torch.equal(a, b)
    dy = torch.randn((T, H), generator=g, device="cuda")
    got = []
    for r, s, v in ((rows, clean, w), (bad_rows, slot_row, bad_w)):
        d_rows, d_w = torch.zeros_like(rows), torch.empty_like(w)
        moe.moe_unpermute_backward(dy, s, d_rows, weights=v, rows=r, d_weights=d_w)
        got.append((d_rows, d_w))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("start,H", [(0, 40), (8, 40), (1, 40), (3, 37), (4, 44)])
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_unpermute_strided_rows(moe, start, H, dtype, out):
    g = gen(start)
    T, K = 70, 3
    wide, dyw = torch.randn((T * K, 64), generator=g, device="cuda").to(dtype), torch.randn((T, 96), generator=g, device="cuda").to(out)
    slot_row, w = slots(g, T, K, 0.1), torch.randn((T, K), generator=g, device="cuda")
    cols = slice(start, start + H)
    yw, dw = torch.full((T, 72), 9.0, device="cuda").to(out), torch.full((T * K, 80), 9.0, device="cuda").to(dtype)
    moe.moe_unpermute(wide[:, cols], slot_row, yw[:, cols], weights=w)
    y = torch.empty((T, H), dtype=out, device="cuda")
    moe.moe_unpermute(wide[:, cols].contiguous(), slot_row, y, weights=w)
    assert torch.equal(y, yw[:, cols]) and (yw[:, :start] == 9).all() and (yw[:, start + H:] == 9).all()
    d_w, d_w2 = torch.empty((T, K), device="cuda"), torch.empty((T, K), device="cuda")
    moe.moe_unpermute_backward(dyw[:, cols], slot_row, dw[:, cols], weights=w, rows=wide[:, cols], d_weights=d_w)
    d_rows = torch.full((T * K, H), 9.0, device="cuda").to(dtype)
    moe.moe_unpermute_backward(dyw[:, cols].contiguous(), slot_row, d_rows, weights=w, rows=wide[:, cols].contiguous(), d_weights=d_w2)
    assert torch.equal(d_rows, dw[:, cols]) and (dw[:, :start] == 9).all() and (dw[:, start + H:] == 9).all()
    terms = (dyw[:, cols].double()[:, None, :] * wide[:, cols].double()[slot_row.clamp_min(0).long()]).abs().sum(-1)
    assert ((d_w - d_w2).abs() <= 2 * (H + 8) * U * terms).all()


def test_there_and_back_with_gradients(moe):
    """A run of the three: the weighted sum of a token's own rows, whose gradients are known in closed form."""
    g = gen(9)
    T, H, E, K = 900, 200, 32, 4
    x, ids = torch.randn((T, H), generator=g, device="cuda"), routes(g, T, E, K, 0.1)
    w = torch.rand((T, K), generator=g, device="cuda")
    rows, out, _, _ = permute(moe, x, ids, E)
    y = torch.empty_like(x)
    moe.moe_unpermute(rows, out["slot_row"], y, weights=w)
    on = (ids >= 0).double()
    total = (w.double() * on).sum(1, keepdim=True)
    assert ((y.double() - total * x.double()).abs() <= (K + 1) * U * (total * x.double()).abs()).all()
    d_rows, d_w, dx = torch.full_like(rows, float("nan")), torch.empty_like(w), torch.empty_like(x)
    dy = torch.randn((T, H), generator=g, device="cuda")
    moe.moe_unpermute_backward(dy, out["slot_row"], d_rows, weights=w, rows=rows, d_weights=d_w)
    moe.moe_unpermute(d_rows, out["slot_row"], dx)  # the gradient of moe_permute
    assert ((dx.double() - total * dy.double()).abs() <= (2 * K + 1) * U * (total * dy.double()).abs()).all()
    dots, size = (x.double() * dy.double()).sum(1, keepdim=True), (x.double() * dy.double()).abs().sum(1, keepdim=True)
    assert ((d_w.double() - dots * on).abs() <= (H + 8) * U * size).all()


def test_row_ops_on_other_streams_and_in_a_graph(moe):
    g = gen(5)
    T, H, E, K = 600, 96, 16, 4
    d = moe.dims(T, 0, 0, E, K)
    x, ids = torch.randn((T, H), generator=g, device="cuda"), routes(g, T, E, K, 0.1)
    w, dy = torch.rand((T, K), generator=g, device="cuda"), torch.randn((T, H), generator=g, device="cuda")
    ws = moe.alloc_ops_workspace(moe.moe_permute_workspace_bytes(d))

    def buffers():
        i = dict(dtype=torch.int32, device="cuda")
        return [torch.zeros((T * K, H), device="cuda"), torch.empty(E + 1, **i), torch.empty(T * K, **i), torch.empty((T, K), **i),
                torch.empty((T, H), device="cuda"), torch.zeros((T * K, H), device="cuda"), torch.empty((T, K), device="cuda")]

    def step(b, stream=None):
        rows, offsets, row_src, slot_row, y, d_rows, d_w = b
        moe.moe_permute(x, ids, d, rows, offsets, row_src, slot_row, ws, stream=stream)
        moe.moe_unpermute(rows, slot_row, y, weights=w, stream=stream)
        moe.moe_unpermute_backward(dy, slot_row, d_rows, weights=w, rows=rows, d_weights=d_w, stream=stream)
    want, other, captured = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(other, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for turn in range(2):
        ids.copy_(routes(g, T, E, K, 0.2))  # the replay sorts the ids that are there then
        for b in captured + want:
            b.zero_()
        graph.replay()
        step(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured))


def test_permute_of_many_slots(moe):
    """More slots than the runs' shortest lengths make up (128 of 1024), a last run that is cut, experts of very different popularity."""
    g = gen(10)
    T, H, E, K = 30011, 4, 200, 7
    ids = (torch.rand((T, K), generator=g, device="cuda") ** 3 * E).to(torch.int32)
    ids[torch.rand((T, K), generator=g, device="cuda") < 0.05] = -1
    x = values(g, T, H, torch.float32)
    rows, out, _, status = permute(moe, x, ids, E)
    flat = ids.flatten().cpu()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    R = int((flat >= 0).sum())
    assert status == moe.MOE_OK and out["offsets"][-1] == R and torch.equal(out["row_src"][:R].cpu().long(), order[:R])
    assert torch.equal(out["offsets"].cpu().long().diff(), torch.bincount(flat[flat >= 0].long(), minlength=E))
    want = torch.full((T * K,), -1, dtype=torch.int64)
    want[order[:R]] = torch.arange(R)
    assert torch.equal(out["slot_row"].flatten().cpu().long(), want) and torch.equal(rows[:R], x[(order[:R] // K).cuda()])


def test_permute_offsets_past_32_bits(moe):
    """Rows whose byte offsets pass 2^32 (and element offsets 2^31)."""
    T, H, K = 70000, 4096, 8  # 560000 rows of 4096 bytes in each of codes: 2.3 GB; of bf16: 4.6 GB
    g = gen(6)
    x = torch.randint(0, 2 ** 15, (T, H), generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    ids = routes(g, T, 4, K)
    rows, out, _, status = permute(moe, x, ids, 4, rows=torch.empty((T * K, H), dtype=torch.bfloat16, device="cuda"))
    assert status == moe.MOE_OK
    token = out["row_src"].long() // K
    assert torch.equal(out["slot_row"].flatten()[out["row_src"].long()], torch.arange(T * K, dtype=torch.int32, device="cuda"))
    for at in range(0, T * K, 40000):
        assert torch.equal(rows[at:at + 40000].view(torch.int16), x[token[at:at + 40000]].view(torch.int16))
    one = torch.ones((T, K), device="cuda")
    y = torch.empty((T, H), dtype=torch.float32, device="cuda")
    rows.fill_(0.25)
    moe.moe_unpermute(rows, out["slot_row"], y, weights=one)
    assert (y == 2.0).all()
    del rows, y
    torch.cuda.empty_cache()
