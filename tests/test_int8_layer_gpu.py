"""The row operators, the quantiser and the grouped INT8 product together, as examples/int8_layer.py uses them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from gpu_util import lib
    lib()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_layer.py")
    spec = importlib.util.spec_from_file_location("int8_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("shape,tokens", [((1024, 512, 32, 4), 150), ((512, 384, 8, 2), 1), ((256, 128, 60, 6), 7), ((1280, 640, 16, 3), 900)])
def test_layer_by_parts_is_the_layer(example, shape, tokens):
    """Both ways round each expert's row to bf16 and the sum to bf16 (2^-8 each, so the difference is within 4 * 2^-8); the one that weighs
    its rows first loses no more. Scales one unit apart in the last place move a code in ten thousand by one step."""
    assert example.compare(example.Layer(*shape), tokens) < 4 * 2.0 ** -8 + 0.004


def test_layer_by_parts_with_masked_routes(example):
    layer = example.Layer(512, 256, 8, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((40, 512), generator=g, device="cuda").to(torch.bfloat16)
    ids, weights = layer.routes(x)
    ids[3] = -1
    ids[5, 1] = ids[39, 0] = -1
    a, b = example.by_parts(layer, x, ids, weights).float(), example.whole(layer, x, ids, weights).float()
    assert (a[3] == 0).all() and (b[3] == 0).all()
    assert (a - b).norm() / b.norm() < 4 * 2.0 ** -8 + 0.004


def test_example_gradients(example):
    """Against torch's differentiation of the plain sum in 64 bits; fp32 products over H and the T rows of an expert."""
    T, H, E, K = 50, 64, 6, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, dy = torch.randn((T, H), generator=g, device="cuda"), torch.randn((T, H), generator=g, device="cuda")
    ids = torch.topk(torch.randn((T, E), generator=g, device="cuda"), K).indices.to(torch.int32).contiguous()
    ids[4, 1], ids[9] = -1, -1
    weights, experts = torch.rand((T, K), generator=g, device="cuda"), torch.randn((E, H, H), generator=g, device="cuda") * H ** -0.5
    got = example.gradients(x, ids, weights, experts, dy)
    leaves = [t.double().requires_grad_(True) for t in (x, weights, experts)]
    on = (ids >= 0).double()
    y = (torch.einsum("th,tkhj->tkj", leaves[0], leaves[2][ids.clamp_min(0).long()]) * (leaves[1] * on)[..., None]).sum(1)
    want = [y, *torch.autograd.grad(y, leaves, dy.double())]
    for a, b in zip(got, want):
        # sums of at most K * H (dx) or T (d_experts) products that are sums of H themselves: 2 * K * H roundings of 2^-24 of magnitudes
        # that stay below 40 here
        assert (a.double() - b).abs().max() <= 2 * K * H * 2.0 ** -24 * 40
