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
