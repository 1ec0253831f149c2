"""moe_int8_quantize and moe_int8_matmul on the GPU against plain implementations. Both are defined to the bit (IEEE divisions and half-even
rounding; an exact integer product, rounded to fp32 and at each product with a scale), so equality is asked for throughout."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------------------
# the quantiser
# ---------------------------------------------------------------------------------------


def quantize_by_definition(x):
    """On the host, fp32 throughout (torch's CPU division is IEEE's)."""
    v = x.float().cpu()
    scale = torch.clamp_min(v.abs().amax(-1) * torch.tensor(1.0 / 127.0), torch.tensor(1e-8))
    return torch.round(v / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 8), (5, 100), (3, 2048), (4, 2056), (7, 4096), (2, 5001), (300, 1536), (3, 7168),
                                 (2, 8192), (2, 8193), (2, 8200), (1, 20000), (2, 40001)])
def test_quantize(moe, M, K, dtype):
    g = gen(M + K)
    x = (torch.randn((M, K), generator=g, device="cuda") * torch.randn((M, 1), generator=g, device="cuda").mul(4).exp()).to(dtype)
    q, scale = torch.full((M, K), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    moe.moe_int8_quantize(x, q, scale)
    want_q, want_scale = quantize_by_definition(x)
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(q.cpu(), want_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1231, 5003])
@pytest.mark.parametrize("K", [1, 3, 4, 8, 16, 24, 40, 61, 72, 129, 248, 256, 264, 511, 512, 520, 1000, 1032, 2048])
def test_quantize_many_short_rows(moe, M, K, dtype):
    """Rows that lanes of a warp have: strided, some of them zeros, infinite or NaN, the largest value anywhere."""
    g = gen(M + K)
    x = torch.randn((M, K + 8), generator=g, device="cuda") * torch.randn((M, 1), generator=g, device="cuda").mul(4).exp()
    x[5::97], x[6::97, K // 2], x[7::97, 0], x[8::97, K - 1] = 0.0, math.inf, -math.inf, math.nan
    x = x.to(dtype)[:, :K]
    q, scale = torch.full((M + 1, K + 16), 99, dtype=torch.int8, device="cuda"), torch.full((M + 1,), -1.0, device="cuda")
    moe.moe_int8_quantize(x, q[:M, :K], scale[:M])
    want_q, want_scale = quantize_by_definition(x)
    finite = want_scale < math.inf  # (the codes of the others are zero)
    want_q[~finite] = 0
    assert torch.equal(scale[:M].cpu().nan_to_num(nan=-2.0), want_scale.nan_to_num(nan=-2.0)) and torch.equal(q[:M, :K].cpu(), want_q)
    assert (q[:, K:] == 99).all() and (q[M] == 99).all() and scale[M] == -1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [64, 61])
def test_quantize_ties_zeros_and_extremes(moe, K, dtype):
    big, small = torch.finfo(dtype).max, 2.0 ** -126
    rows = [[0.0] * K, [-0.0] * K, [127.0] + [0.5, 1.5, 2.5, -0.5, -1.5, -2.5] * 5 + [0.0] * (K - 31), [big] + [-big] * (K - 1),
            [small] * K, [1e-30] * K, [127e-8 * 0.5] + [1e-8] * (K - 1), [big] + [1.0] * (K - 1), [1e-38, -1e-38] + [0.0] * (K - 2),
            [-1.0] + [0.5] * (K - 1), [254.0] + [1.0, 3.0, 5.0, -3.0] * 4 + [7.0] * (K - 17), [2.0 ** 100] + [2.0 ** 99] * (K - 1)]
    x = torch.tensor(rows, dtype=torch.float64).clamp(-big, big).to(dtype).cuda()
    q, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(rows), device="cuda")
    moe.moe_int8_quantize(x, q, scale)
    want_q, want_scale = quantize_by_definition(x)
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(q.cpu(), want_q)
    assert q.min() >= -127


@pytest.mark.parametrize("exponent", [-149, -140, -100, -60, -20, 0, 20, 60, 90, 120])
def test_quantize_quotients_of_any_size(moe, exponent):
    """Random mantissas: quotients that lie near the middle between two codes, at scales from subnormal to near the top."""
    g = gen(exponent + 200)
    x = (torch.randint(-2 ** 24, 2 ** 24, (64, 1000), generator=g, device="cuda").double() * 2.0 ** (exponent - 24 + 7)).float()
    q, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")
    moe.moe_int8_quantize(x, q, scale)
    want_q, want_scale = quantize_by_definition(x)
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(q.cpu(), want_q)


def test_quantize_rows_that_are_not_finite(moe):
    for K in (64, 61, 9000):
        x = torch.ones((4, K), device="cuda")
        x[0, 3], x[1, K - 1], x[2, 0] = math.inf, math.nan, -math.inf
        q, scale = torch.full((4, K), 5, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
        moe.moe_int8_quantize(x, q, scale)
        assert scale[0] == math.inf and scale[1].isnan() and scale[2] == math.inf and (q[:3] == 0).all()
        assert (q[3] == 127).all()


@pytest.mark.parametrize("start", [0, 1, 3, 8])
@pytest.mark.parametrize("K", [40, 43])
def test_quantize_strided_rows(moe, start, K):
    g = gen(start)
    wide = torch.randn((50, 64), generator=g, device="cuda").to(torch.bfloat16)
    q, scale = torch.full((50, 72), 99, dtype=torch.int8, device="cuda"), torch.empty(50, device="cuda")
    moe.moe_int8_quantize(wide[:, start:start + K], q[:, start:start + K], scale)
    want_q, want_scale = quantize_by_definition(wide[:, start:start + K])
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(q[:, start:start + K].cpu(), want_q)
    assert (q[:, :start] == 99).all() and (q[:, start + K:] == 99).all()


# ---------------------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------------------


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def product_by_definition(a, a_scale, b, b_scale, offsets, out):
    """In place into `out` (fp32 or bf16): double holds the integer product exactly."""
    ends = [0, a.shape[0]] if offsets is None else offsets.tolist()
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            c = a[lo:hi].double() @ b[i].double().T
            assert c.abs().max() < 2 ** 31
            out[lo:hi] = ((c.float() * b_scale[i]) * a_scale[lo:hi, None]).to(out.dtype)
    return out


def run(moe, a, a_scale, b, b_scale, offsets, dtype, out=None):
    (M, K), (G, N, _) = a.shape, b.shape
    ws = moe.alloc_ops_workspace(moe.moe_int8_matmul_workspace_bytes(M, N, K, G))
    if out is None:
        out = torch.full((M, N), 9.0, device="cuda").to(dtype)
    moe.moe_int8_matmul(a, a_scale, b, b_scale, out, ws, offsets=offsets)
    assert moe.moe_check_device_error(ws) == moe.MOE_OK
    return out


def case(g, M, N, K, G=1):
    return codes(g, M, K), torch.rand(M, generator=g, device="cuda") + 0.5, codes(g, G, N, K), torch.rand((G, N), generator=g, device="cuda") - 0.5


# row counts around the tiles' edges, from one to many; widths and depths that end inside a tile; depths past an exact fp32 sum
DENSE = [(1, 1, 16), (1, 128, 16), (1, 4096, 7168), (2, 2112, 7168), (3, 100, 1040), (7, 33, 48), (8, 513, 2064), (9, 640, 1024),
         (16, 129, 1008), (17, 300, 4096), (31, 1000, 512), (32, 257, 304), (33, 256, 2048), (64, 130, 3584), (65, 2112, 1552),
         (127, 96, 128), (128, 128, 128), (129, 129, 144), (133, 2112, 7168), (200, 4096, 272), (256, 300, 1040), (257, 511, 1168),
         (300, 256, 20000), (512, 1024, 1024), (700, 1500, 2064), (1000, 2112, 720), (1031, 4100, 1312), (3000, 1111, 256),
         (2048, 4096, 1040), (2, 8, 131056)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_matmul_dense(moe, M, N, K, dtype):
    c = case(gen(M + N + K), M, N, K)
    want = product_by_definition(*c, None, torch.full((M, N), 9.0, device="cuda").to(dtype))
    assert torch.equal(run(moe, *c, None, dtype), want)


@pytest.mark.parametrize("M,N,K", [(1, 256, 7168), (4, 300, 4096), (20, 300, 4096), (40, 300, 4096), (200, 300, 4096), (1200, 1100, 4096),
                                   (3, 16, 131056), (100, 200, 65536), (600, 1024, 65536)])
@pytest.mark.parametrize("low,high", [(-128, -128), (127, 127), (-128, 127), (127, -128)])
def test_matmul_largest_sums(moe, M, N, K, low, high):
    """Codes at their limits in the same direction: partial sums as large as they can be, one code changed so that low bits count."""
    a = torch.full((M, K), low, dtype=torch.int8, device="cuda")
    b = torch.full((1, N, K), high, dtype=torch.int8, device="cuda")
    a[:, K - 1] = (torch.arange(M, device="cuda") % 7 - 3).to(torch.int8)
    b[:, :, K // 2] = (torch.arange(N, device="cuda") % 11 - 5).to(torch.int8)
    one, ones = torch.ones(M, device="cuda"), torch.ones((1, N), device="cuda")
    want = product_by_definition(a, one, b, ones, None, torch.empty((M, N), device="cuda"))
    assert torch.equal(run(moe, a, one, b, ones, None, torch.float32), want)


GROUPED = [([3, 0, 1, 5], 200, 512), ([0, 0, 0], 64, 128), ([1] * 40, 300, 1040), ([0, 130, 128, 1, 127, 0, 64], 384, 2064),
           ([257, 31, 32, 33, 16, 15, 17, 0, 8, 9], 520, 1552), ([700, 0, 900], 1000, 720), ([2000, 1, 1, 1], 256, 1168),
           ([64, 64, 0, 64], 4096, 272), ([0] * 100 + [5] + [0] * 155, 128, 256), ([40] * 32, 1024, 2048), ([4] * 24, 640, 7168),
           ([600, 500, 0, 800], 2112, 1040)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spare", [0, 37])
@pytest.mark.parametrize("counts,N,K", GROUPED)
def test_matmul_grouped(moe, counts, N, K, spare, dtype):
    M = sum(counts) + spare
    if M == 0:
        pytest.skip("no rows")
    c = case(gen(M + N + K), M, N, K, len(counts))
    offsets = torch.tensor([0] + counts, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    want = product_by_definition(*c, offsets, torch.full((M, N), 9.0, device="cuda").to(dtype))
    assert torch.equal(run(moe, *c, offsets, dtype), want)  # rows behind the last group are left alone


def test_matmul_group_offsets_of_any_value(moe):
    """As moe_fp8_matmul takes them: outside [0, M] as the nearest bound, one below an earlier one as that one."""
    M, N, K = 90, 160, 528
    for given, taken in (([0, 40, 30, 200], [0, 40, 40, 90]), ([-5, 10, 10, 50], [0, 10, 10, 50]), ([0, -3, 90, 7], [0, 0, 90, 90])):
        c = case(gen(3), M, N, K, 3)
        want = product_by_definition(*c, torch.tensor(taken), torch.full((M, N), 9.0, device="cuda"))
        got = run(moe, *c, torch.tensor(given, dtype=torch.int32, device="cuda"), torch.float32)
        assert torch.equal(got, want)


def test_matmul_one_group_with_offsets(moe):
    for M, rows in ((50, 33), (4, 4), (700, 0)):
        c = case(gen(M), M, 200, 272, 1)
        offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        want = product_by_definition(*c, offsets, torch.full((M, 200), 9.0, device="cuda"))
        assert torch.equal(run(moe, *c, offsets, torch.float32), want)


@pytest.mark.parametrize("M", [2, 40, 700])
def test_matmul_strided_operands(moe, M):
    g = gen(M)
    N, K = 300, 528
    a_wide, b_wide = codes(g, M, 1024), codes(g, 2, N, 640)
    a, b = a_wide[:, 16:16 + K], b_wide[:, :, 32:32 + K]
    a_scale, b_scale = torch.rand(M, generator=g, device="cuda"), torch.rand((2, N), generator=g, device="cuda")
    offsets = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    for dtype, first in ((torch.bfloat16, 3), (torch.float32, 0), (torch.float32, 1)):
        wide = torch.full((M, 400), 9.0, device="cuda").to(dtype)
        out = wide[:, first:first + N]
        want = product_by_definition(a, a_scale, b, b_scale, offsets, torch.full((M, N), 9.0, device="cuda").to(dtype))
        run(moe, a, a_scale, b, b_scale, offsets, dtype, out=out)
        assert torch.equal(out, want) and (wide[:, :first] == 9).all() and (wide[:, first + N:] == 9).all()


def test_matmul_scales_that_are_not_finite(moe):
    for M in (3, 50, 600):
        a, a_scale, b, b_scale = case(gen(M), M, 140, 160)
        a_scale[1], b_scale[0, 3], b_scale[0, 139] = math.nan, math.inf, -math.inf
        want = product_by_definition(a, a_scale, b, b_scale, None, torch.empty((M, 140), device="cuda"))
        got = run(moe, a, a_scale, b, b_scale, None, torch.float32)
        torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)


def test_matmul_on_other_streams_and_in_a_graph(moe):
    g = gen(8)
    N, K = 520, 1552
    for M in (5, 140, 900):
        c = case(g, M, N, K)
        ws = moe.alloc_ops_workspace(moe.moe_int8_matmul_workspace_bytes(M, N, K, 1))
        want = product_by_definition(*c, None, torch.empty((M, N), device="cuda"))
        torch.cuda.synchronize()
        outs = [torch.empty((M, N), device="cuda") for _ in range(3)]
        sides = [torch.cuda.Stream(), torch.cuda.Stream()]  # two calls at once, a workspace each
        spaces = [ws, moe.alloc_ops_workspace(ws.numel())]
        torch.cuda.synchronize()
        for s, o, w in zip(sides, outs, spaces):
            moe.moe_int8_matmul(*c, o, w, stream=s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_int8_matmul(*c, outs[2], ws)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        c[0].copy_(codes(g, M, K))
        graph.replay()
        assert torch.equal(outs[2], product_by_definition(*c, None, want))


def test_quantize_then_multiply_is_near_the_product(moe):
    """A run of both: each code is off by at most half a step, so a product of K of them by at most the sum of what either side is off."""
    g = gen(11)
    M, N, K = 100, 200, 1024
    x, w = torch.randn((M, K), generator=g, device="cuda"), torch.randn((N, K), generator=g, device="cuda")
    xq, wq = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty((N, K), dtype=torch.int8, device="cuda")
    xs, wscale = torch.empty(M, device="cuda"), torch.empty(N, device="cuda")
    moe.moe_int8_quantize(x, xq, xs)
    moe.moe_int8_quantize(w, wq, wscale)
    y = run(moe, xq, xs, wq[None], wscale[None], None, torch.float32)
    ref = x.double() @ w.double().T
    half_x, half_w = 0.5001 * xs.double()[:, None], 0.5001 * wscale.double()
    bound = half_x * w.abs().double().sum(1) + half_w * x.abs().double().sum(1, keepdim=True) + K * half_x * half_w
    assert ((y.double() - ref).abs() <= bound * 1.0001).all()
