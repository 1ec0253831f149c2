"""moe_int8_matmul on one output of every expert: weights that are a view, whose groups lie apart."""
import pytest
import torch

from test_int8_ops_gpu import gen, product_by_definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from gpu_util import lib
    return lib()


@pytest.mark.parametrize("M", [3, 40, 700, 5000])  # few rows a group, one-CTA tiles, pairs
@pytest.mark.parametrize("G,N,K,at", [(4, 7, 64, 0), (3, 40, 256, 39), (32, 5, 1040, 2)])
def test_one_weight_row_a_group(moe, G, N, K, at, M):
    g = gen(M + G)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda").to(torch.int8)[:, at:at + 1]
    a_scale, w_scale = torch.rand(M, generator=g, device="cuda"), torch.rand((G, 1), generator=g, device="cuda")
    cuts = torch.randint(0, M + 1, (G - 1,), generator=g, device="cuda").sort().values.to(torch.int32)
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), M)])
    out = torch.full((M, 1), 9.0, device="cuda")
    ws = moe.alloc_ops_workspace(moe.moe_int8_matmul_workspace_bytes(M, 1, K, G))
    moe.moe_int8_matmul(a, a_scale, w, w_scale, out, ws, offsets=offsets)
    want = product_by_definition(a, a_scale, w, w_scale, offsets, torch.full((M, 1), 9.0, device="cuda"))
    assert torch.equal(out, want) and moe.moe_check_device_error(ws) == moe.MOE_OK
