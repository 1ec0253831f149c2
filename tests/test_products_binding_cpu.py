"""Row strides that moe_int8_matmul's and moe_fp8_matmul's binding hands to the library. Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import moe_expert_ffn_topk_gb300 as m
    return m


@pytest.fixture
def strides(moe, monkeypatch):
    """Host tensors pass for device memory of one device; the call gives (b_stride, N, groups) instead of reaching the library."""
    b = moe._binding
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(b, "_handle", lambda stream, t: 0)
    seen = []

    class Lib:
        @staticmethod
        def moe_int8_matmul(args, ws, nbytes, stream):
            seen.append((args.b_stride, args.N, args.groups))
            return 0
        moe_fp8_matmul = moe_int8_matmul
    monkeypatch.setattr(b, "LIB", Lib())

    def call(which, weights):
        rows, K = 3, weights.shape[-1]
        G, N = (1, *weights.shape)[-3:-1] if weights.dim() == 2 else weights.shape[:2]
        offsets = torch.zeros(G + 1, dtype=torch.int32) if G > 1 else None
        ws = torch.zeros(256, dtype=torch.uint8)
        if which == "int8":
            moe.moe_int8_matmul(torch.zeros((rows, K), dtype=torch.int8), torch.zeros(rows), weights, torch.zeros(G, N), torch.zeros(rows, N),
                                ws, offsets=offsets)
        else:
            blocks = (K + 127) // 128
            moe.moe_fp8_matmul(torch.zeros((rows, K), dtype=torch.uint8), torch.zeros(rows, blocks), weights.view(torch.uint8),
                               torch.zeros(G, (N + 127) // 128, blocks), torch.zeros(rows, N), ws, offsets=offsets)
        return seen[-1]
    return call


@pytest.mark.parametrize("which", ["int8", "fp8"])
def test_stride_between_weight_rows(strides, which):
    w = torch.zeros((4, 7, 64), dtype=torch.int8)
    assert strides(which, w) == (64, 7, 4)
    assert strides(which, w[..., :32]) == (64, 7, 4)
    assert strides(which, w[0]) == (64, 7, 1) and strides(which, w[2:3]) == (64, 7, 1)
    assert strides(which, w[0, :1]) == (64, 1, 1)
    assert strides(which, torch.zeros((4, 1, 64), dtype=torch.int8)) == (64, 1, 4)


@pytest.mark.parametrize("which", ["int8", "fp8"])
def test_groups_of_one_weight_row_may_lie_apart(strides, which):
    """One output of every expert of a larger matrix: the groups' only rows are as far apart as the groups."""
    w = torch.zeros((4, 7, 64), dtype=torch.int8)
    assert strides(which, w[:, :1]) == (7 * 64, 1, 4)
    assert strides(which, w[:, 3:4, 16:48]) == (7 * 64, 1, 4)
    assert strides(which, w[::2, 6:]) == (14 * 64, 1, 2)
    with pytest.raises(ValueError, match="follow each other"):
        strides(which, w[:, :2])
