"""ctypes binding of the C ABI in ``include/moe_ffn.h``, ``include/moe_ops.h`` and ``include/moe_peak.h``.

Argument marshalling only: each function takes torch tensors (device memory allocated by
the caller), checks placement and contiguity, passes their addresses and the current CUDA
stream to the library function of the same name, and turns a non-OK status into
``MoeError``. Every stage of the computation runs in the library's CUDA kernels. When the
library has not been built, importing this module raises ``ImportError``.
"""
from __future__ import annotations

import ctypes
import os

import torch

# MOE_GB300_DEBUG=1 loads the bounds-checking build (compiled with -DMOE_DEBUG by build(debug=True)):
# the same kernels with every data-dependent row index checked on the device (MOE_ERR_BOUNDS)
_LIB_NAME = "libmoe_gb300_debug.so" if os.environ.get("MOE_GB300_DEBUG") == "1" else "libmoe_gb300.so"
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", _LIB_NAME)

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_BAD_ROUTE, MOE_ERR_TIMEOUT, \
    MOE_ERR_WORKSPACE, MOE_ERR_BAD_SCALE, MOE_ERR_BOUNDS = range(9)
MODES = {"a16w16": 0, "a8w8_fp8": 1, "a8w8_int8": 2, "a8w4_fp8_fp4": 3, "a8w4_int": 4, "a8w8_fp8_e5m2": 5}
(MOE_FLAG_NONE, MOE_FLAG_SIMT, MOE_FLAG_WEIGHT_MAJOR, MOE_FLAG_QUANTIZE_X, MOE_FLAG_FUSED, MOE_FLAG_SINGLE_CTA,
 MOE_FLAG_PAIR_L1, MOE_FLAG_TOKEN_MAJOR, MOE_FLAG_PREPARED_WEIGHTS) = 0, 1, 2, 4, 8, 16, 32, 64, 128

ABI_FUNCTIONS = ("moe_workspace_bytes", "moe_plan", "moe_dispatch", "moe_expert_l1", "moe_expert_l2",
                 "moe_combine", "moe_forward", "moe_check_device_error", "moe_status_string",
                 "moe_workspace_layout", "moe_debug_bounded_wait", "moe_plan_noalloc", "moe_dispatch_quantize",
                 "moe_expert_l1_ex", "moe_forward_ex", "moe_expert_ffn", "moe_tensor_peak_probe",
                 "moe_prepared_weights_bytes", "moe_prepare_weights",
                 "moe_ops_workspace_init", "moe_gate", "moe_fp8_quantize", "moe_fp8_matmul_workspace_bytes",
                 "moe_fp8_matmul", "moe_layer_workspace_bytes", "moe_layer")
# moe_peak_kind (include/moe_peak.h): the tcgen05 instruction kinds the probe measures
PEAK_KINDS = {"bf16": 0, "f16": 1, "e4m3_e2m1": 2, "e4m3_e4m3": 3}
# moe_ops.h: element types, router scores, weight formats of moe_layer
MOE_TYPE_BF16, MOE_TYPE_F32 = 0, 1
SCORES = {"softmax": 0, "sigmoid": 1}
LAYER_WEIGHTS = {"bf16": 0, "fp8_block": 1, "fp4_mx": 2}
MOE_QUANT_POW2 = 1
MOE_LAYER_MAX_TOKENS = 64


class MoeDims(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("num_shared_experts", ctypes.c_int32)]


class MoeOptions(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("has_activation_clamp", ctypes.c_uint32),
                ("activation_clamp", ctypes.c_float)]


class MoeOperand(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class MoeWorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "header", "counts", "offsets", "pad_offsets", "tile_offsets", "row_src", "pool_src", "slot_row", "gates",
        "x_pool", "x_pool_scale", "a_pool", "a_pool_scale", "a_f32", "x_pool_planes", "a_pool_planes", "pool_sums",
        "comb", "ffn_counters",
        "total")] + \
        [("pool_rows", ctypes.c_int64)]


class MoeGateOptions(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("normalize", ctypes.c_int32), ("route_scale", ctypes.c_float)]


class MoeFp8MatmulArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("a", "a_scale", "b", "b_scale", "offsets", "out")] + \
        [(n, ctypes.c_int64) for n in ("M", "N", "K", "a_stride", "b_stride", "out_stride")] + \
        [("groups", ctypes.c_int32), ("out_type", ctypes.c_int32)]


class MoeLayerArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("router", ctypes.c_void_p), ("w1", MoeOperand), ("w2", MoeOperand),
                ("gate", ctypes.POINTER(MoeGateOptions)), ("gate_bias", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
                ("topk_weights", ctypes.c_void_p), ("y", ctypes.c_void_p), ("router_type", ctypes.c_int32),
                ("weights", ctypes.c_int32), ("has_activation_clamp", ctypes.c_uint32), ("activation_clamp", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {moe_status_string(status)} (status {status})")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"CUDA library not built ({_LIB_PATH} is missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, sz, u32, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int
    dims_p = ctypes.POINTER(MoeDims)
    sig = {
        "moe_workspace_bytes": (sz, [dims_p, st]),
        "moe_plan": (st, [vp, dims_p, vp, vp, vp, vp, sz, vp]),
        "moe_dispatch": (st, [MoeOperand, dims_p, st, vp, sz, vp]),
        "moe_expert_l1": (st, [MoeOperand, dims_p, st, u32, vp, sz, vp]),
        "moe_expert_l2": (st, [MoeOperand, vp, dims_p, st, u32, vp, sz, vp]),
        "moe_combine": (st, [vp, dims_p, vp, sz, vp]),
        "moe_forward": (st, [MoeOperand, vp, vp, MoeOperand, MoeOperand, vp, dims_p, st, u32, vp, sz, vp]),
        "moe_check_device_error": (st, [vp, vp]),
        "moe_status_string": (ctypes.c_char_p, [st]),
        "moe_workspace_layout": (st, [dims_p, st, ctypes.POINTER(MoeWorkspaceLayout)]),
        "moe_debug_bounded_wait": (st, [vp, sz, ctypes.c_uint64, vp]),
        "moe_plan_noalloc": (st, [vp, dims_p, vp, vp, vp, vp]),
        "moe_dispatch_quantize": (st, [vp, dims_p, st, vp, sz, vp]),
        "moe_expert_l1_ex": (st, [MoeOperand, dims_p, st, ctypes.POINTER(MoeOptions), vp, sz, vp]),
        "moe_expert_ffn": (st, [MoeOperand, MoeOperand, vp, vp, dims_p, st, ctypes.POINTER(MoeOptions), vp, sz, vp]),
        "moe_forward_ex": (st, [MoeOperand, vp, vp, MoeOperand, MoeOperand, vp, dims_p, st, ctypes.POINTER(MoeOptions),
                                vp, sz, vp]),
        "moe_tensor_peak_probe": (st, [st, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_double), vp, sz, vp]),
        "moe_prepared_weights_bytes": (sz, [dims_p, st, ctypes.c_int]),
        "moe_prepare_weights": (st, [vp, dims_p, st, ctypes.c_int, vp, sz, vp]),
        "moe_ops_workspace_init": (st, [vp, sz, vp]),
        "moe_gate": (st, [vp, st, ctypes.c_int64, vp, ctypes.POINTER(MoeGateOptions), dims_p, vp, vp, vp]),
        "moe_fp8_quantize": (st, [vp, st, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_int64, vp, u32, vp]),
        "moe_fp8_matmul_workspace_bytes": (sz, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
        "moe_fp8_matmul": (st, [ctypes.POINTER(MoeFp8MatmulArgs), vp, sz, vp]),
        "moe_layer_workspace_bytes": (sz, [dims_p, st]),
        "moe_layer": (st, [ctypes.POINTER(MoeLayerArgs), dims_p, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


LIB = _load()


# ---------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------


def dims(T: int, H: int, I: int, E: int, K: int, S: int = 0) -> MoeDims:  # noqa: E741
    """T tokens, hidden H, intermediate I, E routed experts, top-K, S shared experts."""
    return MoeDims(T, H, I, E, K, S)


def _mode(m) -> int:
    return MODES[m] if isinstance(m, str) else int(m)


def _ptr(t, what, dev=True):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if dev and not t.is_cuda:
        raise ValueError(f"{what} must be in device memory")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr() if t.numel() else None


def _operand(data, scale, what):
    return MoeOperand(_ptr(data, what), _ptr(scale, what + "_scale"))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ws(workspace):
    return _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


# ---------------------------------------------------------------------------------------
# the ABI, one function each
# ---------------------------------------------------------------------------------------


def moe_status_string(status: int) -> str:
    return LIB.moe_status_string(int(status)).decode()


def moe_workspace_bytes(d: MoeDims, mode) -> int:
    return LIB.moe_workspace_bytes(ctypes.byref(d), _mode(mode))


def moe_workspace_layout(d: MoeDims, mode) -> dict:
    out = MoeWorkspaceLayout()
    _check(LIB.moe_workspace_layout(ctypes.byref(d), _mode(mode), ctypes.byref(out)), "moe_workspace_layout")
    return {name: getattr(out, name) for name, _ in MoeWorkspaceLayout._fields_}


def moe_plan(topk_ids, d: MoeDims, workspace, counts=None, offsets=None, row_src=None, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_plan(_ptr(topk_ids, "topk_ids"), ctypes.byref(d), _ptr(counts, "counts"),
                        _ptr(offsets, "offsets"), _ptr(row_src, "row_src"), ws, nb, _stream(stream)), "moe_plan")


def moe_dispatch(x, x_scale, d: MoeDims, mode, workspace, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_dispatch(_operand(x, x_scale, "x"), ctypes.byref(d), _mode(mode), ws, nb, _stream(stream)),
           "moe_dispatch")


def moe_dispatch_quantize(x_bf16, d: MoeDims, mode, workspace, stream=None):
    """S2 from bf16 x with the mode's activation quantisation (x_bf16: bf16 [T, H])."""
    ws, nb = _ws(workspace)
    _check(LIB.moe_dispatch_quantize(_ptr(x_bf16, "x_bf16"), ctypes.byref(d), _mode(mode), ws, nb, _stream(stream)),
           "moe_dispatch_quantize")


def moe_expert_l1(w1, w1_scale, d: MoeDims, mode, workspace, flags=0, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_expert_l1(_operand(w1, w1_scale, "w1"), ctypes.byref(d), _mode(mode), flags, ws, nb,
                             _stream(stream)), "moe_expert_l1")


def moe_expert_l2(w2, w2_scale, topk_weights, d: MoeDims, mode, workspace, flags=0, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_expert_l2(_operand(w2, w2_scale, "w2"), _ptr(topk_weights, "topk_weights"), ctypes.byref(d),
                             _mode(mode), flags, ws, nb, _stream(stream)), "moe_expert_l2")


def moe_combine(y, d: MoeDims, workspace, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_combine(_ptr(y, "y"), ctypes.byref(d), ws, nb, _stream(stream)), "moe_combine")


def moe_forward(x, x_scale, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, y, d: MoeDims, mode, workspace,
                flags=0, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_forward(_operand(x, x_scale, "x"), _ptr(topk_ids, "topk_ids"), _ptr(topk_weights, "topk_weights"),
                           _operand(w1, w1_scale, "w1"), _operand(w2, w2_scale, "w2"), _ptr(y, "y"),
                           ctypes.byref(d), _mode(mode), flags, ws, nb, _stream(stream)), "moe_forward")


def _options(flags, activation_clamp):
    return MoeOptions(int(flags), 0 if activation_clamp is None else 1,
                      0.0 if activation_clamp is None else float(activation_clamp))


def moe_expert_l1_ex(w1, w1_scale, d: MoeDims, mode, workspace, flags=0, activation_clamp=None, stream=None):
    """moe_expert_l1 with options (activation_clamp: None or >= 0)."""
    ws, nb = _ws(workspace)
    opt = _options(flags, activation_clamp)
    _check(LIB.moe_expert_l1_ex(_operand(w1, w1_scale, "w1"), ctypes.byref(d), _mode(mode), ctypes.byref(opt), ws, nb,
                                _stream(stream)), "moe_expert_l1_ex")


def moe_expert_ffn(w1, w1_scale, w2, w2_scale, topk_weights, d: MoeDims, mode, workspace, y=None,
                   activation_clamp=None, stream=None):
    """S3-S5 (and S6 into y when given) in one launch with dependency counters; needs
    moe_dispatch first."""
    ws, nb = _ws(workspace)
    opt = _options(0, activation_clamp)
    _check(LIB.moe_expert_ffn(_operand(w1, w1_scale, "w1"), _operand(w2, w2_scale, "w2"),
                              _ptr(topk_weights, "topk_weights"), None if y is None else _ptr(y, "y"), ctypes.byref(d),
                              _mode(mode), ctypes.byref(opt), ws, nb, _stream(stream)), "moe_expert_ffn")


def moe_forward_ex(x, x_scale, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, y, d: MoeDims, mode, workspace,
                   flags=0, activation_clamp=None, stream=None):
    """moe_forward with options (activation_clamp: None or >= 0)."""
    ws, nb = _ws(workspace)
    opt = _options(flags, activation_clamp)
    _check(LIB.moe_forward_ex(_operand(x, x_scale, "x"), _ptr(topk_ids, "topk_ids"), _ptr(topk_weights, "topk_weights"),
                              _operand(w1, w1_scale, "w1"), _operand(w2, w2_scale, "w2"), _ptr(y, "y"),
                              ctypes.byref(d), _mode(mode), ctypes.byref(opt), ws, nb, _stream(stream)),
           "moe_forward_ex")


def moe_check_device_error(workspace, stream=None) -> int:
    return LIB.moe_check_device_error(_ptr(workspace, "workspace"), _stream(stream))


def moe_debug_bounded_wait(workspace, timeout_ns: int, stream=None):
    ws, nb = _ws(workspace)
    _check(LIB.moe_debug_bounded_wait(ws, nb, int(timeout_ns), _stream(stream)), "moe_debug_bounded_wait")


def moe_prepared_weights_bytes(d: MoeDims, mode, layer: int) -> int:
    return LIB.moe_prepared_weights_bytes(ctypes.byref(d), _mode(mode), int(layer))


def moe_prepare_weights(w, d: MoeDims, mode, layer: int, out=None, stream=None):
    """The layer's weights in the prepared form the GEMMs take with MOE_FLAG_PREPARED_WEIGHTS (A8W8-INT:
    every int8 code as its exact f16 value, same layout); writes `out` (allocated here when None) and
    returns it."""
    n = moe_prepared_weights_bytes(d, mode, layer)
    if out is None:
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED if _mode(mode) != MODES["a8w8_int8"] else MOE_ERR_INVALID_ARG,
                           "moe_prepare_weights")
        out = torch.empty(w.shape, dtype=torch.float16, device=w.device)  # the same layout as the int8 codes
    _check(LIB.moe_prepare_weights(_ptr(w, "w"), ctypes.byref(d), _mode(mode), int(layer), _ptr(out, "out"),
                                   out.numel() * out.element_size(), _stream(stream)), "moe_prepare_weights")
    return out


def moe_tensor_peak_probe(kind, iters_per_cta: int, workspace, grid: int = 0, stream=None) -> float:
    """Launches the dense tensor-core probe of one instruction kind ("bf16", "f16", "e4m3_e2m1",
    "e4m3_e4m3"); returns the flops the launch performs (time it with events on `stream`)."""
    ws, nb = _ws(workspace)
    flops = ctypes.c_double(0.0)
    k = PEAK_KINDS[kind] if isinstance(kind, str) else int(kind)
    _check(LIB.moe_tensor_peak_probe(k, int(iters_per_cta), int(grid), ctypes.byref(flops), ws, nb, _stream(stream)),
           "moe_tensor_peak_probe")
    return flops.value


def moe_plan_noalloc(topk_ids, d: MoeDims, counts, offsets, row_src, stream=None):
    """moe_plan without a workspace (its scratch is a fixed device array inside the library)."""
    _check(LIB.moe_plan_noalloc(_ptr(topk_ids, "topk_ids"), ctypes.byref(d), _ptr(counts, "counts"),
                                _ptr(offsets, "offsets"), _ptr(row_src, "row_src"), _stream(stream)),
           "moe_plan_noalloc")


# ---------------------------------------------------------------------------------------
# include/moe_ops.h: the router, the block-scaled FP8 product, the few-token layer
# ---------------------------------------------------------------------------------------


_FLOAT_TYPES = {torch.bfloat16: MOE_TYPE_BF16, torch.float32: MOE_TYPE_F32}
_FP8_CODES = (torch.float8_e4m3fn, torch.uint8)
# the current device, and its current stream's handle without a Stream object around it (a third of a small call's host time otherwise)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, t):
    """Handle of `stream`, or of the current stream. The library launches on the current device, so t has to be there."""
    device = t.get_device()
    if device != _current_device():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(device)


def _vec(t, what, dtype, shape):
    """Address of a contiguous device tensor of that type (or of one of a tuple of them) and shape."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be in device memory")
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _float_type(t, what):
    try:
        return _FLOAT_TYPES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be bfloat16 or float32") from None


def _rows(t, what, shape):
    """Row stride of a device matrix of that shape whose rows are contiguous (a column slice of a wider one is)."""
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be in device memory")
    stride, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    return stride if shape[0] > 1 else shape[1]


def _space(workspace):
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous device memory")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def moe_ops_workspace_init(workspace, stream=None):
    ws, nb = _space(workspace)
    _check(LIB.moe_ops_workspace_init(ws, nb, _handle(stream, workspace)), "moe_ops_workspace_init")


def gate_options(score="softmax", groups=1, topk_groups=1, group_top=1, normalize=True, route_scale=1.0) -> MoeGateOptions:
    """Options of the router: score "softmax" or "sigmoid"; the experts in `groups` equal runs of which the `topk_groups`
    with the largest sum of their `group_top` (1 or 2) best choice values stay; normalised weights; their scale."""
    return MoeGateOptions(SCORES[score], int(groups), int(topk_groups), int(group_top), int(bool(normalize)), float(route_scale))


def moe_gate(logits, d: MoeDims, topk_ids, topk_weights, bias=None, options=None, stream=None):
    """topk_ids (int32 [T,K]) and topk_weights (fp32 [T,K]) from logits (bf16 or fp32 [T,E], rows may be strided)."""
    T, E, K = d.num_tokens, d.num_experts, d.topk
    status = LIB.moe_gate(logits.data_ptr(), _float_type(logits, "logits"), _rows(logits, "logits", (T, E)),
                          None if bias is None else _vec(bias, "bias", torch.float32, (E,)), options, d,
                          _vec(topk_ids, "topk_ids", torch.int32, (T, K)),
                          _vec(topk_weights, "topk_weights", torch.float32, (T, K)), _handle(stream, logits))
    if status:
        raise MoeError(status, "moe_gate")


def moe_fp8_quantize(x, q, scale, pow2=False, stream=None):
    """Rows of x (bf16 or fp32 [M,K]) into q (e4m3 [M,K]) and scale (fp32 [M, ceil(K/128)]); rows of x and q may be strided."""
    M, K = shape = x.shape
    if q.dtype not in _FP8_CODES:
        raise TypeError("q must be float8_e4m3fn or uint8")
    status = LIB.moe_fp8_quantize(x.data_ptr(), _float_type(x, "x"), M, K, _rows(x, "x", shape), q.data_ptr(), _rows(q, "q", shape),
                                  _vec(scale, "scale", torch.float32, (M, (K + 127) // 128)), MOE_QUANT_POW2 if pow2 else 0,
                                  _handle(stream, x))
    if status:
        raise MoeError(status, "moe_fp8_quantize")


def moe_fp8_matmul_workspace_bytes(M: int, N: int, K: int, groups: int = 1) -> int:
    return LIB.moe_fp8_matmul_workspace_bytes(M, N, K, groups)


def moe_fp8_matmul(a, a_scale, b, b_scale, out, workspace, offsets=None, stream=None):
    """out[m,n] = sum over blocks of a_scale * b_scale * (a . b^T): a e4m3 [M,K], a_scale fp32 [M, ceil(K/128)], b e4m3
    [groups,N,K] (or [N,K]), b_scale fp32 [groups, ceil(N/128), ceil(K/128)], out bf16 or fp32 [M,N]. With `offsets`
    (int32 [groups+1]) rows [offsets[g], offsets[g+1]) are multiplied by b[g]. Rows of a, b and out may be strided."""
    if a.dtype not in _FP8_CODES or b.dtype not in _FP8_CODES:
        raise TypeError("a and b must be float8_e4m3fn (or uint8 codes)")
    shape = a.shape
    M, K = shape
    kb = (K + 127) // 128
    if b.dim() == 3:
        G, N, k2 = b.shape
        between, b_stride, one = b.stride()
        if G > 1 and between != N * b_stride:
            raise ValueError("the groups of b must follow each other")
        b_scale_shape = (G, (N + 127) // 128, kb)
        if b_scale.dim() == 2 and G == 1:
            b_scale_shape = b_scale_shape[1:]
    else:
        G, (N, k2), (b_stride, one) = 1, b.shape, b.stride()
        b_scale_shape = ((N + 127) // 128, kb) if b_scale.dim() == 2 else (1, (N + 127) // 128, kb)
    if k2 != K or not b.is_cuda or one != 1:
        raise ValueError(f"b must be device memory of {K} contiguous columns")
    if G * N == 1:
        b_stride = K
    ws, nbytes = _space(workspace)
    args = MoeFp8MatmulArgs(a.data_ptr(), _vec(a_scale, "a_scale", torch.float32, (M, kb)), b.data_ptr(),
                            _vec(b_scale, "b_scale", torch.float32, b_scale_shape),
                            None if offsets is None else _vec(offsets, "offsets", torch.int32, (G + 1,)), out.data_ptr(), M, N, K,
                            _rows(a, "a", shape), b_stride, _rows(out, "out", (M, N)), G, _float_type(out, "out"))
    status = LIB.moe_fp8_matmul(args, ws, nbytes, _handle(stream, a))
    if status:
        raise MoeError(status, "moe_fp8_matmul")


# types of moe_layer's weights and of their scales, where the format has any (one-byte codes and scale exponents also as uint8),
# and how many of K's values share a byte, and a scale with how many outputs
_LAYER_TYPES = {
    "bf16": (torch.bfloat16, None, 1, 0, 0),
    "fp8_block": (_FP8_CODES, torch.float32, 1, 128, 128),
    "fp4_mx": (tuple(t for t in (torch.uint8, getattr(torch, "float4_e2m1fn_x2", None)) if t),
               tuple(t for t in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if t), 2, 1, 32),
}


def _layer_operand(data, scale, what, weights, experts, n, k):
    """One of moe_layer's weights, [experts, n, k] with its scales, or bf16 [experts, k, n] (a scale is not read then)."""
    codes, scales, packed, rows, cols = _LAYER_TYPES[weights]
    if data is None or (scale is None and scales is not None):
        raise ValueError(f"{what} of {weights} weights is a tensor{' with its scales' if scales else ''}")
    if scales is None:
        return MoeOperand(_vec(data, what, codes, (experts, k, n)), None)
    return MoeOperand(_vec(data, what, codes, (experts, n, k // packed)),
                      _vec(scale, what + "_scale", scales, (experts, n // rows, k // cols)))


def moe_layer_workspace_bytes(d: MoeDims, weights) -> int:
    return LIB.moe_layer_workspace_bytes(ctypes.byref(d), LAYER_WEIGHTS[weights])


def moe_layer(x, router, w1, w1_scale, w2, w2_scale, y, d: MoeDims, weights, workspace, options=None, bias=None,
              topk_ids=None, topk_weights=None, activation_clamp=None, stream=None):
    """The whole layer for up to MOE_LAYER_MAX_TOKENS tokens in one launch: router product, selection, experts, combine.
    weights: "bf16", "fp8_block" or "fp4_mx"; w1, w2 and their scales in the shapes moe_ops.h lists for it, the shared experts after
    the routed ones. Without a router, topk_ids and topk_weights are inputs; with one they are
    optional outputs."""
    T, H, E, K = d.num_tokens, d.hidden, d.num_experts, d.topk
    args = MoeLayerArgs()
    args.x = _vec(x, "x", torch.bfloat16, (T, H))
    args.y = _vec(y, "y", torch.bfloat16, (T, H))
    args.weights = LAYER_WEIGHTS[weights]
    experts, inter = E + d.num_shared_experts, d.intermediate
    args.w1 = _layer_operand(w1, w1_scale, "w1", weights, experts, 2 * inter, H)
    args.w2 = _layer_operand(w2, w2_scale, "w2", weights, experts, H, inter)
    if router is not None:
        args.router_type = _float_type(router, "router")
        args.router = _vec(router, "router", router.dtype, (E, H))
    if options is not None:
        args.gate = ctypes.pointer(options)
    if bias is not None:
        args.gate_bias = _vec(bias, "bias", torch.float32, (E,))
    if topk_ids is not None:
        args.topk_ids = _vec(topk_ids, "topk_ids", torch.int32, (T, K))
    if topk_weights is not None:
        args.topk_weights = _vec(topk_weights, "topk_weights", torch.float32, (T, K))
    if activation_clamp is not None:
        args.has_activation_clamp, args.activation_clamp = 1, float(activation_clamp)
    ws, nb = _space(workspace)
    status = LIB.moe_layer(args, d, ws, nb, _handle(stream, x))
    if status:
        raise MoeError(status, "moe_layer")
