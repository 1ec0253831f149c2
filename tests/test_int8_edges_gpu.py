"""moe_int8_matmul and the row operators at the calls that the other tests do not make: sums that leave fp32's integers in a part of a tile,
first calls inside a capture, workspaces shared by graphs, every kernel of the product on the same numbers."""
import os
import subprocess
import sys

import pytest
import torch

from test_int8_ops_gpu import case, codes, gen, product_by_definition, run

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


@pytest.mark.parametrize("M,N,K", [(40, 200, 5120), (100, 200, 5120), (300, 2112, 5120), (1100, 1100, 5120), (700, 1500, 40960)])
@pytest.mark.parametrize("big", [0, 17, 33, 47])
def test_sums_that_grow_past_2_24_in_some_tokens(moe, M, N, K, big):
    """Small codes, but for every 48th token from `big` on and every 31st weight row, whose codes are all at the limit: their sums pass 2^24
    after a few chunks of K while the rest stay small, and low bits count on both sides of it."""
    g = gen(big + M)
    a = torch.randint(-9, 10, (M, K), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    b = torch.randint(-9, 10, (1, N, K), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    a[big % M::48] = 127
    b[:, 5::31] = -128
    a[:, ::7] += (torch.arange(M, device="cuda") % 3 - 1).to(torch.int8)[:, None].clamp(max=0)
    one, ones = torch.ones(M, device="cuda"), torch.ones((1, N), device="cuda")
    want = product_by_definition(a, one, b, ones, None, torch.empty((M, N), device="cuda"))
    assert want.abs().max() > 2 ** 24
    assert torch.equal(run(moe, a, one, b, ones, None, torch.float32), want)


def test_rows_do_not_depend_on_the_kernel(moe):
    """A row's result is the same in a product of few rows, of some and of many, and as a group of its own."""
    g = gen(7)
    N, K = 1200, 3088
    a, a_scale, b, b_scale = case(g, 3000, N, K)
    whole = run(moe, a, a_scale, b, b_scale, None, torch.bfloat16)
    for first, rows in ((0, 1), (5, 3), (100, 7), (200, 16), (300, 40), (400, 100), (600, 300), (1000, 900)):
        at = slice(first, first + rows)
        assert torch.equal(run(moe, a[at], a_scale[at], b, b_scale, None, torch.bfloat16), whole[at])
    ends = torch.tensor([0, 2, 2, 19, 300, 3000], dtype=torch.int32, device="cuda")
    many = b.expand(5, N, K).contiguous(), b_scale.expand(5, N).contiguous()
    assert torch.equal(run(moe, a, a_scale, *many, ends, torch.bfloat16), whole)


def test_many_groups(moe):
    """As many groups as the call takes, few of them with rows; and groups that lie past 2^31 bytes of weights."""
    g = gen(12)
    G, N, K = 1024, 256, 512
    counts = torch.zeros(G, dtype=torch.int64)
    counts[[0, 3, 700, 1000, 1023]] = torch.tensor([1, 40, 300, 17, 129])
    offsets = torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    c = case(g, int(counts.sum()), N, K, G)
    want = product_by_definition(*c, offsets, torch.empty((c[0].shape[0], N), device="cuda"))
    assert torch.equal(run(moe, *c, offsets, torch.float32), want)
    G, N, K = 20, 16384, 7168  # 2.3 GB
    counts = torch.tensor([3] + [0] * 17 + [5, 130])
    offsets = torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    M = int(counts.sum())
    b = torch.empty((G, N, K), dtype=torch.int8, device="cuda")
    b.random_(-128, 128, generator=g)
    a, a_scale, b_scale = codes(g, M, K), torch.rand(M, generator=g, device="cuda"), torch.rand((G, N), generator=g, device="cuda")
    want = product_by_definition(a, a_scale, b, b_scale, offsets, torch.empty((M, N), device="cuda"))
    assert torch.equal(run(moe, a, a_scale, b, b_scale, offsets, torch.float32), want)
    few = torch.tensor([0] + [0] * 18 + [7, 7], dtype=torch.int32, device="cuda")  # (of few rows a group: another kernel)
    want = product_by_definition(a[:7], a_scale[:7], b, b_scale, few, torch.empty((7, N), device="cuda"))
    assert torch.equal(run(moe, a[:7], a_scale[:7], b, b_scale, few, torch.float32), want)


def test_long_output_rows(moe):
    """An output whose rows lie past 2^32 bytes apart from the first."""
    g = gen(13)
    M, N, K = 1500, 200, 272
    c = case(g, M, N, K)
    wide = torch.empty(M * (1 << 21), dtype=torch.bfloat16, device="cuda").view(M, 1 << 21)  # 6.3 GB
    out = wide[:, 1000:1000 + N]
    want = product_by_definition(*c, None, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(run(moe, *c, None, torch.bfloat16, out=out), want)
    del wide, out
    torch.cuda.empty_cache()


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, {root!r})
import moe_expert_ffn_topk_gb300 as moe
i32 = dict(dtype=torch.int32, device="cuda")
T, H, E, K, N = 800, 128, 16, 4, 640
x = torch.randn((T, H), device="cuda")
ids = torch.randint(0, E, (T, K), **i32)
d = moe.dims(T, 0, 0, E, K)
q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
rows, row_scale = torch.zeros((T * K, H), dtype=torch.int8, device="cuda"), torch.zeros((T * K, 1), device="cuda")
offsets, row_src, slot_row = torch.empty(E + 1, **i32), torch.empty(T * K, **i32), torch.empty((T, K), **i32)
b, bs = torch.randint(-127, 128, (E, N, H), device="cuda").to(torch.int8), torch.rand((E, N), device="cuda")
w = torch.rand((T, K), device="cuda")
out, y = torch.zeros((T * K, N), device="cuda"), torch.zeros((T, N), device="cuda")
one, dense = torch.zeros((1, N), device="cuda"), torch.zeros((700, N), device="cuda")
ws = moe.alloc_ops_workspace(max(moe.moe_permute_workspace_bytes(d), moe.moe_int8_matmul_workspace_bytes(T * K, N, H, E)))

def step():
    moe.moe_int8_quantize(x, q, s)
    moe.moe_permute(q, ids, d, rows, offsets, row_src, slot_row, ws, scale=s[:, None], row_scale=row_scale)
    moe.moe_int8_matmul(rows, row_scale[:, 0], b, bs, out, ws, offsets=offsets)
    moe.moe_unpermute(out, slot_row, y, weights=w)
    moe.moe_int8_matmul(q[:1], s[:1], b[0], bs[0], one, ws)
    moe.moe_int8_matmul(q[:700], s[:700], b[0], bs[0], dense, ws)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()  # every kernel's first launch in this process
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (rows, out, y, one, dense)]
for t in (rows, out, y, one, dense):
    t.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, c) for a, c in zip(got, (rows, out, y, one, dense)))
other = torch.cuda.CUDAGraph()
with torch.cuda.graph(other):
    step()
for turn in range(3):  # two graphs with one workspace, one after the other
    x.mul_(0.5)
    graph.replay()
    other.replay()
torch.cuda.synchronize()
assert moe.moe_check_device_error(ws) == 0
assert y.isfinite().all() and not torch.equal(y, got[2])
print("first calls ok")
"""


def test_first_calls_inside_a_capture(moe):
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls ok" in r.stdout, r.stderr[-2000:]
