"""Host-side behaviour of the operators of include/moe_ops.h: argument checks, limits and workspace sizes. Nothing is
launched: every call here is refused, or has no work."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import moe_expert_ffn_topk_gb300 as m
    return m


P = ctypes.c_void_p(4096)   # an aligned address; never read
ODD = ctypes.c_void_p(4097)


def gate(moe, d=(4, 128, 128, 16, 2), type=1, stride=16, opt=None, logits=P, ids=P, weights=P, bias=None):
    o = moe.gate_options(**opt) if isinstance(opt, dict) else opt
    return moe._binding.LIB.moe_gate(logits, type, stride, bias, None if o is None else ctypes.byref(o),
                                     ctypes.byref(moe.dims(*d)), ids, weights, None)


@pytest.mark.parametrize("bad", [
    dict(d=(-1, 128, 128, 16, 2)), dict(d=(4, 128, 128, 16, 0)), dict(d=(4, 128, 128, 16, 17)),
    dict(d=(4, 128, 128, 2000, 2)), dict(d=(4, 128, 128, 64, 33)), dict(d=(1 << 23, 128, 128, 16, 4)), dict(type=2), dict(stride=15),
    dict(logits=None), dict(ids=None), dict(weights=None), dict(logits=ODD), dict(bias=ODD),
    dict(opt=dict(groups=3)), dict(opt=dict(groups=0)), dict(opt=dict(groups=4, topk_groups=5)),
    dict(opt=dict(groups=16, topk_groups=1)), dict(opt=dict(groups=4, topk_groups=2, group_top=3)),
    dict(opt=dict(route_scale=float("inf"))), dict(opt=dict(route_scale=float("nan")))])
def test_gate_refuses(moe, bad):
    assert gate(moe, **bad) == moe.MOE_ERR_INVALID_ARG


def test_gate_with_no_tokens(moe):
    assert gate(moe, d=(0, 128, 128, 16, 2), logits=None, ids=None, weights=None) == moe.MOE_OK


def quantize(moe, type=0, rows=4, cols=256, xs=256, qs=256, x=P, q=P, scale=P, flags=0):
    return moe._binding.LIB.moe_fp8_quantize(x, type, rows, cols, xs, q, qs, scale, flags, None)


@pytest.mark.parametrize("bad", [dict(type=3), dict(rows=-1), dict(cols=-1), dict(cols=0), dict(xs=255), dict(qs=255),
                                 dict(x=None), dict(q=None), dict(scale=None), dict(x=ODD), dict(scale=ODD), dict(flags=2),
                                 dict(rows=1 << 62, cols=8, xs=8, qs=8)])
def test_quantize_refuses(moe, bad):
    assert quantize(moe, **bad) == moe.MOE_ERR_INVALID_ARG


def test_quantize_of_nothing(moe):
    assert quantize(moe, rows=0, x=None, q=None, scale=None) == moe.MOE_OK


def matmul(moe, ws=P, ws_bytes=1 << 40, **kw):
    a = dict(a=4096, a_scale=4096, b=4096, b_scale=4096, offsets=None, out=4096, M=4, N=256, K=256, a_stride=256, b_stride=256,
             out_stride=256, groups=1, out_type=0)
    a.update(kw)
    args = moe._binding.MoeFp8MatmulArgs(*[a[n] for n, _ in moe._binding.MoeFp8MatmulArgs._fields_])
    return moe._binding.LIB.moe_fp8_matmul(ctypes.byref(args), ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=8), dict(K=250), dict(groups=0),
    dict(groups=2), dict(groups=1025, offsets=4096), dict(a_stride=128), dict(b_stride=240), dict(a_stride=264),
    dict(b_stride=264), dict(out_stride=255), dict(out_type=7), dict(a=None), dict(a_scale=None), dict(b=None), dict(b_scale=None),
    dict(out=None), dict(a=4104), dict(b=4104), dict(a_scale=4098), dict(b_scale=4098), dict(out=4097), dict(offsets=4098),
    dict(M=(1 << 31) - 1, a_stride=1 << 40)])
def test_matmul_refuses(moe, bad):
    assert matmul(moe, **bad) == moe.MOE_ERR_INVALID_ARG


def test_matmul_workspace(moe):
    need = moe.moe_fp8_matmul_workspace_bytes(4, 256, 256)
    assert need >= 256
    for ws, have in ((None, need), (ctypes.c_void_p(4104), need), (P, need - 1)):
        assert matmul(moe, ws=ws, ws_bytes=have) == moe.MOE_ERR_WORKSPACE
    for bad in ((-1, 256, 256, 1), (4, 0, 256, 1), (4, 256, 8, 1), (4, 256, 257, 1), (4, 256, 256, 0)):
        assert moe.moe_fp8_matmul_workspace_bytes(*bad) == 0
    assert matmul(moe, M=0, a=None, a_scale=None, out=None, ws=None) == moe.MOE_OK


def layer(moe, d=(4, 256, 128, 8, 2), ws=P, ws_bytes=1 << 40, w1=(4096, 4096), w2=(4096, 4096), gate=None, **kw):
    b = moe._binding
    a = dict(x=4096, router=4096, w1=b.MoeOperand(*w1), w2=b.MoeOperand(*w2),
             gate=None if gate is None else ctypes.pointer(moe.gate_options(**gate)), gate_bias=None, topk_ids=None,
             topk_weights=None, y=4096, router_type=0, weights=1, has_activation_clamp=0, activation_clamp=0.0)
    a.update(kw)
    args = b.MoeLayerArgs(*[a[n] for n, _ in b.MoeLayerArgs._fields_])
    return b.LIB.moe_layer(ctypes.byref(args), ctypes.byref(moe.dims(*d)), ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(d=(4, 100, 128, 8, 2)), dict(d=(4, 256, 96, 8, 2)), dict(d=(4, 256, 128, 8, 30, 3)), dict(d=(-1, 256, 128, 8, 2)),
    dict(weights=3), dict(weights=-1), dict(x=None), dict(y=None), dict(x=4104), dict(router=4104), dict(w1=(None, 4096)),
    dict(w2=(4096, None)), dict(w1=(4104, 4096)), dict(w2=(4096, 4100)), dict(router=None), dict(router=None, topk_ids=4096),
    dict(router_type=2), dict(gate=dict(groups=3)), dict(has_activation_clamp=1, activation_clamp=-1.0),
    dict(has_activation_clamp=1, activation_clamp=float("nan")), dict(topk_ids=4097), dict(gate_bias=4097)])
def test_layer_refuses(moe, bad):
    assert layer(moe, **bad) == moe.MOE_ERR_INVALID_ARG


def test_layer_limits_and_workspace(moe):
    most = moe.MOE_LAYER_MAX_TOKENS
    assert layer(moe, d=(most + 1, 256, 128, 8, 2)) == moe.MOE_ERR_UNSUPPORTED
    for weights in moe.LAYER_WEIGHTS:
        need = moe.moe_layer_workspace_bytes(moe.dims(4, 256, 128, 8, 2, 1), weights)
        assert need > 0 and need >= moe.moe_layer_workspace_bytes(moe.dims(4, 256, 128, 8, 2), weights)
        assert moe.moe_layer_workspace_bytes(moe.dims(most + 1, 256, 128, 8, 2), weights) == 0
        assert moe.moe_layer_workspace_bytes(moe.dims(4, 250, 128, 8, 2), weights) == 0
    need = moe.moe_layer_workspace_bytes(moe.dims(4, 256, 128, 8, 2), "fp8_block")
    for ws, have in ((None, need), (ctypes.c_void_p(4104), need), (P, need - 1)):
        assert layer(moe, ws=ws, ws_bytes=have) == moe.MOE_ERR_WORKSPACE
    assert layer(moe, d=(0, 256, 128, 8, 2), x=None, y=None, ws=None) == moe.MOE_OK
    assert moe._binding.LIB.moe_ops_workspace_init(None, 256, None) == moe.MOE_ERR_WORKSPACE
    assert moe._binding.LIB.moe_ops_workspace_init(ctypes.c_void_p(4104), 256, None) == moe.MOE_ERR_WORKSPACE


def test_binding_checks_shapes_types_and_devices(moe):
    d = moe.dims(4, 256, 128, 8, 2)
    host = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        moe.moe_gate(host, d, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        moe.moe_fp8_quantize(torch.zeros((4, 256)), torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2)))
    with pytest.raises(TypeError):
        moe.moe_fp8_matmul(host, host, host, host, host, host)
    with pytest.raises(ValueError):
        moe.moe_layer(host, None, None, None, None, None, host, d, "bf16", host)
    with pytest.raises(ValueError):
        moe.alloc_ops_workspace(0, "cpu")


def test_header_is_a_c_abi(moe, tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "ops.c"
    src.write_text('#include "moe_ops.h"\n#include <stdio.h>\nint main(void) {\n'
                   '    printf("%zu %zu %zu", sizeof(moe_layer_args), sizeof(moe_fp8_matmul_args), sizeof(moe_gate_options));\n'
                   '    return 0;\n}\n')
    exe = tmp_path / "ops"
    cc = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(root, "include"),
                         str(src), "-o", str(exe)], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    b = moe._binding
    sizes = [ctypes.sizeof(s) for s in (b.MoeLayerArgs, b.MoeFp8MatmulArgs, b.MoeGateOptions)]
    assert [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()] == sizes
