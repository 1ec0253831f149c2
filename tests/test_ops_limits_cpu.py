"""Limits of the calls of include/moe_ops.h where a size meets the width of the kernels' integers. Nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import moe_expert_ffn_topk_gb300 as m
    return m


@pytest.mark.parametrize("past", [1, 100, 256, 511])
def test_matmul_rows_stay_inside_32_bits(moe, past):
    """Groups may begin at any row and a tile has 256: past 2^31 - 512 rows the last tile's row numbers could wrap."""
    most = (1 << 31) - 512
    assert moe.moe_fp8_matmul_workspace_bytes(most, 1, 16, 2) > 0
    assert moe.moe_fp8_matmul_workspace_bytes(most + past, 1, 16, 2) == 0
    fields = dict(a=4096, a_scale=4096, b=4096, b_scale=4096, offsets=4096, out=4096, M=most + past, N=1, K=16, a_stride=16, b_stride=16,
                  out_stride=1, groups=2, out_type=1)
    args = moe._binding.MoeFp8MatmulArgs(*[fields[n] for n, _ in moe._binding.MoeFp8MatmulArgs._fields_])
    # (without a workspace, so that no version of the library gets as far as a launch)
    assert moe._binding.LIB.moe_fp8_matmul(ctypes.byref(args), None, 0, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", ["bf16", "fp8_block", "fp4_mx"])
@pytest.mark.parametrize("sizes", [(6528, 640, 256, 3, 2), (3712, 15104, 60, 1, 2), (1664, 6144, 60, 2, 1), (2944, 12032, 64, 2, 2),
                                   (4224, 5632, 60, 5, 2), (7168, 2048, 256, 8, 1), (128, 16384, 1, 1, 0)])
def test_a_layer_workspace_serves_fewer_tokens(moe, fmt, sizes):
    """Fewer tokens can cut K into more parts; a workspace for the most tokens of a server takes them all the same."""
    need = [moe.moe_layer_workspace_bytes(moe.dims(t, *sizes), fmt) for t in range(65)]
    assert all(n > 0 for n in need) and need == sorted(need)
