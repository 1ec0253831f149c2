"""One workspace, zeroed once, that several operators of moe_ops.h use in turn: every call leaves the counters at zero for the next one, whichever
operator that is. What the definition fixes is asked for bit for bit."""
import pytest
import torch

from test_ops_gpu import FORMATS, gen, layer_weights, randn, run_layer
from test_row_ops_gpu import routes, sort_by_definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


class Permute:
    """A call of moe_permute on a workspace of the caller's, and what it has to give."""

    def __init__(self, moe, g, T, E, K, H=64, masked=0.1):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.moe, self.d = moe, moe.dims(T, 0, 0, E, K)
        self.x, self.ids = torch.randn((T, H), generator=g, device="cuda"), routes(g, T, E, K, masked)
        self.rows = torch.full((T * K, H), 7.0, device="cuda")
        self.offsets, self.row_src, self.slot_row = torch.empty(E + 1, **i32), torch.empty(T * K, **i32), torch.empty((T, K), **i32)
        self.want = sort_by_definition(self.ids, E)
        self.bytes = moe.moe_permute_workspace_bytes(self.d)

    def __call__(self, ws):
        self.moe.moe_permute(self.x, self.ids, self.d, self.rows, self.offsets, self.row_src, self.slot_row, ws)

    def check(self):
        offsets, src, row = self.want
        assert self.offsets.tolist() == offsets and self.row_src.tolist() == src and self.slot_row.flatten().tolist() == row
        routed = offsets[-1]
        token = torch.tensor(src[:routed], device="cuda") // self.d.topk
        assert torch.equal(self.rows[:routed], self.x[token]) and (self.rows[routed:] == 7).all()


# one launch up to 4096 slots (and 2^22 ids counted by its CTAs), sorted runs past that
@pytest.mark.parametrize("T,E,K", [(7, 256, 8), (1, 1, 1), (512, 1024, 8), (513, 1024, 8), (513, 3, 8), (4099, 1, 1), (8192, 256, 8),
                                   (5001, 1000, 31), (200000, 64, 1)])
def test_permute_leaves_its_workspace_at_zero(moe, T, E, K):
    call = Permute(moe, gen(T), T, E, K, H=4)
    ws = moe.alloc_ops_workspace(call.bytes + 4096)
    for _ in range(2):
        call(ws)
        assert int(ws.count_nonzero()) == 0
    call.check()
    call.ids[0, 0] = E  # names no expert: the error word is set, and nothing else
    call(ws)
    assert int(ws[256:].count_nonzero()) == 0
    assert moe.moe_check_device_error(ws) == moe.MOE_ERR_BAD_ROUTE


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I,E,K,S", [(5, 384, 256, 60, 6, 0), (64, 512, 384, 32, 4, 1), (1, 1024, 128, 8, 2, 1)])
def test_layer_after_permute_and_products(moe, fmt, T, H, I, E, K, S):  # noqa: E741
    g = gen(T + H)
    d = moe.dims(T, H, I, E, K, S)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, fmt, E + S, 2 * I, H), layer_weights(g, fmt, E + S, H, I)
    permutes = [Permute(moe, g, *shape) for shape in ((8192, 256, 8), (600, 1024, 8), (9, 40, 4))]
    rows, groups, N, k = 700, 5, 264, 256
    a, b = (torch.randint(-128, 128, shape, generator=g, device="cuda").to(torch.int8) for shape in ((rows, k), (groups, N, k)))
    a_scale, b_scale = torch.rand(rows, generator=g, device="cuda"), torch.rand((groups, N), generator=g, device="cuda")
    offsets = torch.tensor([0, 100, 100, 650, 651, 700], dtype=torch.int32, device="cuda")
    out, alone = torch.empty((rows, N), device="cuda"), torch.empty((rows, N), device="cuda")
    nbytes = max([moe.moe_layer_workspace_bytes(d, fmt), moe.moe_int8_matmul_workspace_bytes(rows, N, k, groups)] + [p.bytes for p in permutes])
    want, status = run_layer(moe, x, router, w1, w2, d, fmt)  # on a workspace of its own
    assert status == moe.MOE_OK
    moe.moe_int8_matmul(a, a_scale, b, b_scale, alone, moe.alloc_ops_workspace(nbytes), offsets=offsets)
    ws = moe.alloc_ops_workspace(nbytes)
    for turn in range(6):
        permutes[turn % 3](ws)
        y, status = run_layer(moe, x, router, w1, w2, d, fmt, ws)
        assert status == moe.MOE_OK and torch.equal(y, want)
        out.zero_()
        moe.moe_int8_matmul(a, a_scale, b, b_scale, out, ws, offsets=offsets)
        assert torch.equal(out, alone)
    for p in permutes:
        p.check()


def test_layer_after_permute_in_one_graph(moe):
    T, H, I, E, K = 4, 256, 128, 16, 2  # noqa: E741
    g = gen(3)
    d = moe.dims(T, H, I, E, K)
    x, router = randn(g, T, H).to(torch.bfloat16), (randn(g, E, H) * H ** -0.5).to(torch.bfloat16)
    w1, w2 = layer_weights(g, "fp8_block", E, 2 * I, H), layer_weights(g, "fp8_block", E, H, I)
    want, _ = run_layer(moe, x, router, w1, w2, d, "fp8_block")
    p = Permute(moe, g, 1100, 128, 4)
    ws = moe.alloc_ops_workspace(max(p.bytes, moe.moe_layer_workspace_bytes(d, "fp8_block")))
    y = torch.empty_like(x)

    def step():
        p(ws)
        moe.moe_layer(x, router, w1[0], w1[1], w2[0], w2[1], y, d, "fp8_block", ws)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
            step()
    for _ in range(4):
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert moe.moe_check_device_error(ws) == moe.MOE_OK
    p.check()
