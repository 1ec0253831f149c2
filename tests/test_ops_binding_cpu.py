"""What the Python binding of include/moe_ops.h refuses before it calls the library: the kernels take the sizes from the dims, so a
tensor of another shape or type would be read past its end."""
import pytest

torch = pytest.importorskip("torch")

T, H, I, E, K, S = 2, 256, 128, 4, 2, 1  # noqa: E741
X = E + S


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import moe_expert_ffn_topk_gb300 as m
    return m


def weights_of(fmt):
    """w1, its scale, w2, its scale as moe_ops.h has them."""
    if fmt == "bf16":
        return [torch.zeros((X, H, 2 * I), dtype=torch.bfloat16), None, torch.zeros((X, I, H), dtype=torch.bfloat16), None]
    if fmt == "fp8_block":
        return [torch.zeros((X, 2 * I, H), dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros((X, 2 * I // 128, H // 128)),
                torch.zeros((X, H, I), dtype=torch.uint8), torch.zeros((X, H // 128, I // 128))]
    u8 = dict(dtype=torch.uint8)
    return [torch.zeros((X, 2 * I, H // 2), **u8), torch.zeros((X, 2 * I, H // 32), **u8), torch.zeros((X, H, I // 2), **u8),
            torch.zeros((X, H, I // 32), **u8)]


@pytest.fixture
def placed(monkeypatch):
    """Host tensors pass for device memory; nothing reads them."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)


@pytest.mark.parametrize("fmt", ["bf16", "fp8_block", "fp4_mx"])
@pytest.mark.parametrize("which", [0, 2])
def test_layer_refuses_weights_of_other_shapes_and_types(moe, placed, fmt, which):
    def refused(error, match, **change):
        w = weights_of(fmt)
        for i, v in change.items():
            w[int(i[1:])] = v(w[int(i[1:])])
        b = moe._binding
        with pytest.raises(error, match=match):
            if which == 0:
                b._layer_operand(w[0], w[1], "w1", fmt, X, 2 * I, H)
            else:
                b._layer_operand(w[2], w[3], "w2", fmt, X, H, I)
    name, scale = f"w{which}", f"w{which + 1}"
    refused(ValueError, "is a tensor", **{name: lambda t: None})
    refused(ValueError, "shape", **{name: lambda t: t[:E]})                       # without the shared expert
    refused(ValueError, "shape", **{name: lambda t: t.transpose(1, 2).contiguous()[:, :, :64]})
    refused(ValueError, "shape", **{name: lambda t: t.flatten(0, 1)})
    refused(TypeError, "must be", **{name: lambda t: torch.zeros(t.shape, dtype=torch.float16)})
    if fmt == "bf16":
        return
    refused(ValueError, "with its scales", **{scale: lambda t: None})
    refused(ValueError, "shape", **{scale: lambda t: t[:E]})
    refused(ValueError, "shape", **{scale: lambda t: t[:, :1]})
    refused(TypeError, "must be", **{scale: lambda t: t.to(torch.float64)})


def test_layer_checks_its_weights_before_the_call(moe, placed, monkeypatch):
    """The whole call, with device placement taken for granted: the library is reached with the declared weights alone."""
    b = moe._binding
    reached = []
    monkeypatch.setattr(b, "_handle", lambda stream, t: 0)
    monkeypatch.setattr(b, "_space", lambda w: (w.data_ptr(), w.numel()))

    class Lib:
        @staticmethod
        def moe_layer(*a):
            reached.append(a)
            return 0
    monkeypatch.setattr(b, "LIB", Lib)
    x, y = torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros((T, H), dtype=torch.bfloat16)
    router, ws, d = torch.zeros((E, H)), torch.zeros(256, dtype=torch.uint8), moe.dims(T, H, I, E, K, S)
    for fmt in ("bf16", "fp8_block", "fp4_mx"):
        w = weights_of(fmt)
        moe.moe_layer(x, router, w[0], w[1], w[2], w[3], y, d, fmt, ws)
        for i in (0, 2) if fmt == "bf16" else range(4):
            short = [t[:E] if j == i else t for j, t in enumerate(w)]
            with pytest.raises(ValueError, match="shape"):
                moe.moe_layer(x, router, short[0], short[1], short[2], short[3], y, d, fmt, ws)
    assert len(reached) == 3


def test_tensors_of_another_device_than_the_current_one_are_refused(moe, placed, monkeypatch):
    """The library launches on the calling thread's device; a stream or pointers of another one do not belong there."""
    b = moe._binding
    reached = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: reached.append(name) or 0
    monkeypatch.setattr(b, "LIB", Lib())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(b, "_raw_stream", lambda device: 0)

    class Stream:
        cuda_stream = 0
    d = moe.dims(T, H, I, E, K, S)
    x, q = torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros((T, H), dtype=torch.uint8)
    scale, ids, ws = torch.zeros((T, H // 128)), torch.zeros((T, K), dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    w = weights_of("fp8_block")
    calls = {
        "moe_gate": lambda **k: moe.moe_gate(torch.zeros((T, E)), d, ids, torch.zeros((T, K)), **k),
        "moe_fp8_quantize": lambda **k: moe.moe_fp8_quantize(x, q, scale, **k),
        "moe_fp8_matmul": lambda **k: moe.moe_fp8_matmul(q, scale, torch.zeros((128, H), dtype=torch.uint8), torch.zeros((1, H // 128)),
                                                         torch.zeros((T, 128)), ws, **k),
        "moe_layer": lambda **k: moe.moe_layer(x, torch.zeros((E, H)), *w, x.clone(), d, "fp8_block", ws, **k),
        "moe_ops_workspace_init": lambda **k: moe.moe_ops_workspace_init(ws, **k),
    }
    for current in (0, 1):
        monkeypatch.setattr(b, "_current_device", lambda: current, raising=False)
        for name, call in calls.items():
            for stream in (None, Stream()):
                reached.clear()
                if current == 1:
                    call(stream=stream)
                    assert reached == [name]
                else:
                    with pytest.raises(ValueError, match="current device"):
                        call(stream=stream)
                    assert reached == []
