"""What moe_permute, moe_unpermute, moe_unpermute_backward, moe_int8_quantize and moe_int8_matmul refuse, in the library and in the binding
before it. Nothing is launched: every call is refused on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

P = 4096  # an address no call gets as far as using
INVALID, WORKSPACE = 1, 6


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import moe_expert_ffn_topk_gb300 as m
    return m


def permute(moe, T=4, K=2, E=8, ws=P, nbytes=1 << 20, **change):
    fields = dict(x=P, scale=None, topk_ids=P, rows=P, row_scale=None, offsets=P, row_src=P, slot_row=P, H=64, x_stride=64, rows_stride=64,
                  type=0, scales=0)
    fields.update(change)
    b = moe._binding
    args = b.MoePermuteArgs(*[fields[n] for n, _ in b.MoePermuteArgs._fields_])
    return b.LIB.moe_permute(ctypes.byref(args), ctypes.byref(moe.dims(T, 0, 0, E, K)), ws, nbytes, None)


@pytest.mark.parametrize("change", [
    dict(K=0), dict(K=33), dict(E=0), dict(E=1025), dict(T=-1), dict(T=1 << 20, K=32), dict(H=0), dict(H=(1 << 30) + 1, x_stride=1 << 31),
    dict(x_stride=63), dict(rows_stride=63), dict(x_stride=1 << 62), dict(type=3), dict(type=-1), dict(x=None), dict(topk_ids=None),
    dict(rows=None), dict(offsets=None), dict(row_src=None), dict(slot_row=None), dict(x=P + 1), dict(rows=P + 1), dict(x=P + 2, type=1),
    dict(offsets=P + 2), dict(row_src=P + 2), dict(slot_row=P + 2), dict(topk_ids=P + 2), dict(scale=P, scales=1),
    dict(scale=P, row_scale=P, scales=-1), dict(scale=P, row_scale=P, scales=(1 << 20) + 1), dict(scale=P + 2, row_scale=P, scales=1)])
def test_permute_refuses(moe, change):
    assert permute(moe, **change) == INVALID


def test_permute_workspace(moe):
    d = moe.dims(4, 0, 0, 8, 2)
    assert moe.moe_permute_workspace_bytes(d) == 256
    assert permute(moe, ws=None) == WORKSPACE and permute(moe, ws=P + 16) == WORKSPACE and permute(moe, nbytes=255) == WORKSPACE
    for K in (1, 2, 7, 8, 32):  # enough for fewer tokens, too
        need = [moe.moe_permute_workspace_bytes(moe.dims(T, 0, 0, 64, K)) for T in range(1, 4200)]
        assert need == sorted(need) and need[-1] == 256 + 4 * 128 * 64
    for bad in ((4, 0, 0, 0, 2), (4, 0, 0, 8, 33), (-1, 0, 0, 8, 2), (1 << 23, 0, 0, 8, 4)):
        assert moe.moe_permute_workspace_bytes(moe.dims(*bad)) == 0
    with pytest.raises(ValueError):
        moe.alloc_ops_workspace(0, "cpu")


def unpermute(moe, T=4, K=2, **change):
    f = dict(rows=P, type=0, rows_stride=64, slot_row=P, weights=P, H=64, y=P, y_type=1, y_stride=64)
    f.update(change)
    return moe._binding.LIB.moe_unpermute(f["rows"], f["type"], f["rows_stride"], f["slot_row"], f["weights"],
                                          ctypes.byref(moe.dims(T, 0, 0, 0, K)), f["H"], f["y"], f["y_type"], f["y_stride"], None)


@pytest.mark.parametrize("change", [
    dict(K=0), dict(K=33), dict(T=-1), dict(T=1 << 20, K=32), dict(H=0), dict(H=65), dict(rows_stride=63), dict(y_stride=63), dict(type=2),
    dict(y_type=2), dict(type=-1), dict(rows=None), dict(slot_row=None), dict(y=None), dict(rows=P + 1), dict(y=P + 2), dict(weights=P + 2),
    dict(slot_row=P + 1), dict(rows_stride=1 << 62)])
def test_unpermute_refuses(moe, change):
    assert unpermute(moe, **change) == INVALID


def test_unpermute_of_no_tokens(moe):
    assert unpermute(moe, T=0, rows=None, slot_row=None, y=None) == 0


def backward(moe, T=4, K=2, **change):
    f = dict(dy=P, dy_type=1, dy_stride=64, rows=P, type=0, rows_stride=64, slot_row=P, weights=P, H=64, d_rows=P, d_rows_stride=64,
             d_weights=P)
    f.update(change)
    return moe._binding.LIB.moe_unpermute_backward(f["dy"], f["dy_type"], f["dy_stride"], f["rows"], f["type"], f["rows_stride"],
                                                   f["slot_row"], f["weights"], ctypes.byref(moe.dims(T, 0, 0, 0, K)), f["H"],
                                                   f["d_rows"], f["d_rows_stride"], f["d_weights"], None)


@pytest.mark.parametrize("change", [
    dict(K=0), dict(K=33), dict(T=-1), dict(H=0), dict(dy_stride=63), dict(rows_stride=63), dict(d_rows_stride=63), dict(type=2),
    dict(dy_type=2), dict(dy=None), dict(rows=None), dict(slot_row=None), dict(d_rows=None), dict(dy=P + 2), dict(rows=P + 1),
    dict(d_rows=P + 1), dict(d_weights=P + 1), dict(weights=P + 1), dict(slot_row=P + 2)])
def test_unpermute_backward_refuses(moe, change):
    assert backward(moe, **change) == INVALID


def quantize(moe, **change):
    f = dict(x=P, type=0, rows=4, cols=64, x_stride=64, q=P, q_stride=64, scale=P)
    f.update(change)
    return moe._binding.LIB.moe_int8_quantize(f["x"], f["type"], f["rows"], f["cols"], f["x_stride"], f["q"], f["q_stride"], f["scale"], None)


@pytest.mark.parametrize("change", [
    dict(type=2), dict(type=-1), dict(rows=-1), dict(cols=-1), dict(cols=0), dict(cols=65), dict(x_stride=63), dict(q_stride=63),
    dict(cols=(1 << 30) + 1, x_stride=1 << 31, q_stride=1 << 31), dict(x=None), dict(q=None), dict(scale=None), dict(x=P + 1),
    dict(x=P + 2, type=1), dict(scale=P + 2), dict(x_stride=1 << 61)])
def test_quantize_refuses(moe, change):
    assert quantize(moe, **change) == INVALID


def test_quantize_of_no_rows(moe):
    assert quantize(moe, rows=0, cols=0, x=None, q=None, scale=None) == 0


def matmul(moe, ws=P, nbytes=1 << 20, **change):
    f = dict(a=P, a_scale=P, b=P, b_scale=P, offsets=None, out=P, M=8, N=64, K=128, a_stride=128, b_stride=128, out_stride=64, groups=1,
             out_type=0)
    f.update(change)
    b = moe._binding
    args = b.MoeInt8MatmulArgs(*[f[n] for n, _ in b.MoeInt8MatmulArgs._fields_])
    return b.LIB.moe_int8_matmul(ctypes.byref(args), ws, nbytes, None)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(M=(1 << 31) - 511, groups=2, offsets=P), dict(N=0), dict(N=(1 << 20) + 1, out_stride=1 << 21), dict(K=0),
    dict(K=136, a_stride=144, b_stride=144), dict(K=1 << 17, a_stride=1 << 17, b_stride=1 << 17), dict(groups=0), dict(groups=1025, offsets=P),
    dict(groups=2), dict(a_stride=112), dict(b_stride=112), dict(out_stride=63), dict(a_stride=136), dict(b_stride=136), dict(a=None),
    dict(a_scale=None), dict(b=None), dict(b_scale=None), dict(out=None), dict(a=P + 8), dict(b=P + 8), dict(a_scale=P + 2),
    dict(b_scale=P + 2), dict(offsets=P + 2), dict(out=P + 1), dict(out=P + 2, out_type=1), dict(out_type=2), dict(a_stride=1 << 62)])
def test_matmul_refuses(moe, change):
    assert matmul(moe, **change) == INVALID


def test_matmul_workspace_and_no_rows(moe):
    assert moe.moe_int8_matmul_workspace_bytes(8, 64, 131056, 1) > 0 and moe.moe_int8_matmul_workspace_bytes(8, 64, 131072, 1) == 0
    assert moe.moe_int8_matmul_workspace_bytes(8, 64, 136, 1) == 0
    assert matmul(moe, ws=None) == WORKSPACE and matmul(moe, ws=P + 128) == WORKSPACE and matmul(moe, nbytes=8) == WORKSPACE
    assert matmul(moe, M=0, ws=None, a=None) == 0


# ---------------------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------------------


@pytest.fixture
def placed(moe, monkeypatch):
    """Host tensors pass for device memory of one device; a call that reaches the library is an error of the test."""
    b = moe._binding
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(b, "_handle", lambda stream, t: 0)

    class Lib:
        def __getattr__(self, name):
            def reached(*a):
                raise AssertionError(f"{name} was called")
            return reached
    monkeypatch.setattr(b, "LIB", Lib())


def test_binding_of_permute_refuses(moe, placed):
    T, H, E, K = 3, 8, 4, 2
    i32 = dict(dtype=torch.int32)
    good = dict(x=torch.zeros(T, H), topk_ids=torch.zeros((T, K), **i32), d=moe.dims(T, 0, 0, E, K), rows=torch.zeros(T * K, H),
                offsets=torch.zeros(E + 1, **i32), row_src=torch.zeros(T * K, **i32), slot_row=torch.zeros((T, K), **i32),
                workspace=torch.zeros(256, dtype=torch.uint8))
    for error, change in ((TypeError, dict(x=torch.zeros(T, H, dtype=torch.float16))), (TypeError, dict(rows=torch.zeros(T * K, H).bfloat16())),
                          (ValueError, dict(rows=torch.zeros(T, H))), (ValueError, dict(x=torch.zeros(T + 1, H))),
                          (ValueError, dict(rows=torch.zeros(H, T * K).T)), (TypeError, dict(topk_ids=torch.zeros((T, K), dtype=torch.int64))),
                          (ValueError, dict(offsets=torch.zeros(E, **i32))), (ValueError, dict(row_src=torch.zeros(T, **i32))),
                          (ValueError, dict(slot_row=torch.zeros(T * K, **i32))), (ValueError, dict(scale=torch.zeros(T, 1))),
                          (ValueError, dict(scale=torch.zeros(T, 1), row_scale=torch.zeros(T, 1))),
                          (TypeError, dict(scale=torch.zeros(T, 1).double(), row_scale=torch.zeros(T * K, 1)))):
        with pytest.raises(error):
            moe.moe_permute(**{**good, **change})
    with pytest.raises(AssertionError, match="moe_permute was called"):
        moe.moe_permute(**good)


def test_binding_of_unpermute_refuses(moe, placed):
    T, H, K = 3, 8, 2
    good = dict(rows=torch.zeros(T * K, H), slot_row=torch.zeros((T, K), dtype=torch.int32), y=torch.zeros(T, H), weights=torch.zeros(T, K))
    for error, change in ((TypeError, dict(rows=torch.zeros(T * K, H, dtype=torch.int8))), (ValueError, dict(rows=torch.zeros(T * K, H + 1))),
                          (TypeError, dict(slot_row=torch.zeros((T, K), dtype=torch.int64))), (ValueError, dict(weights=torch.zeros(T * K))),
                          (TypeError, dict(weights=torch.zeros(T, K).bfloat16())), (ValueError, dict(y=torch.zeros(T + 1, H))),
                          (TypeError, dict(y=torch.zeros(T, H).half())), (ValueError, dict(y=torch.zeros(H, T).T))):
        with pytest.raises(error):
            moe.moe_unpermute(**{**good, **change})
    with pytest.raises(AssertionError, match="moe_unpermute was called"):
        moe.moe_unpermute(**good)
    good = dict(dy=torch.zeros(T, H), slot_row=good["slot_row"], d_rows=torch.zeros(T * K, H), weights=torch.zeros(T, K),
                rows=torch.zeros(T * K, H), d_weights=torch.zeros(T, K))
    for error, change in ((ValueError, dict(rows=None)), (ValueError, dict(d_weights=None)), (TypeError, dict(d_rows=torch.zeros(T * K, H).bfloat16())),
                          (ValueError, dict(d_rows=torch.zeros(T, H))), (ValueError, dict(d_weights=torch.zeros(T * K))),
                          (ValueError, dict(dy=torch.zeros(T, H + 1))), (ValueError, dict(dy=torch.zeros(1, 1).expand(T, H)))):
        with pytest.raises(error):
            moe.moe_unpermute_backward(**{**good, **change})
    with pytest.raises(AssertionError, match="moe_unpermute_backward was called"):
        moe.moe_unpermute_backward(**good)


def test_binding_of_int8_refuses(moe, placed):
    i8 = dict(dtype=torch.int8)
    good = dict(x=torch.zeros(3, 32), q=torch.zeros((3, 32), **i8), scale=torch.zeros(3))
    for error, change in ((TypeError, dict(x=torch.zeros(3, 32).half())), (TypeError, dict(q=torch.zeros(3, 32, dtype=torch.uint8))),
                          (ValueError, dict(q=torch.zeros((3, 31), **i8))), (ValueError, dict(scale=torch.zeros(3, 1)))):
        with pytest.raises(error):
            moe.moe_int8_quantize(**{**good, **change})
    with pytest.raises(AssertionError, match="moe_int8_quantize was called"):
        moe.moe_int8_quantize(**good)
    good = dict(a=torch.zeros((3, 32), **i8), a_scale=torch.zeros(3), b=torch.zeros((2, 5, 32), **i8), b_scale=torch.zeros(2, 5),
                out=torch.zeros(3, 5), workspace=torch.zeros(256, dtype=torch.uint8), offsets=torch.zeros(3, dtype=torch.int32))
    for error, change in ((TypeError, dict(a=torch.zeros(3, 32))), (TypeError, dict(b=torch.zeros(2, 5, 32))), (ValueError, dict(a_scale=torch.zeros(3, 1))),
                          (ValueError, dict(b=torch.zeros((2, 5, 48), **i8))), (ValueError, dict(b_scale=torch.zeros(10))),
                          (ValueError, dict(b=torch.zeros((4, 5, 32), **i8)[::2])), (ValueError, dict(offsets=torch.zeros(2, dtype=torch.int32))),
                          (TypeError, dict(out=torch.zeros(3, 5).half())), (ValueError, dict(out=torch.zeros(5, 3).T))):
        with pytest.raises(error):
            moe.moe_int8_matmul(**{**good, **change})
    with pytest.raises(AssertionError, match="moe_int8_matmul was called"):
        moe.moe_int8_matmul(**good)
