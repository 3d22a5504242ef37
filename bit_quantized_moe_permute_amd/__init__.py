"""Routed 2-bit MoE FFN layer for AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI in include/moe2bit.h (libmoe2bit.so, built
in-tree by build.py).  The functions below have the C names and only marshal
arguments: torch tensors are passed as device pointers, the stream is torch's
current HIP stream, and every step of the layer runs in the library's HIP
kernels.  There is no fallback: if the library is missing or fails to load,
importing the binding raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe2bit.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_DEVICE = 0, 1, 2, 3
DT_F32, DT_BF16, DT_E4M3_BLOCK, DT_E4M3_ROW, DT_F16 = 0, 1, 2, 3, 4
FMT_IQ2X, FMT_Q2K, FMT_Q4K = 1, 2, 3
PATH_AUTO, PATH_GENERIC, PATH_GEMV, PATH_GEMM = 0, 1, 2, 3
PRECISION_EXACT, PRECISION_FAST = 0, 1
ACT_NONE, ACT_SWIGLU = 0, 1
ABI_VERSION = 5
NORM_MAX_HIDDEN = 32768

EXPORTS = [
    "moe_abi_version", "moe_sync_debug", "moe_last_error", "moe_weight_bytes", "moe_prepare_weights",
    "moe_dequantize", "moe_route_workspace", "moe_route", "moe_expert_ffn_workspace", "moe_expert_ffn",
    "moe_expert_gate_up", "moe_expert_down", "moe_combine", "moe_combine_steer", "moe_probe_stream_read",
    "moe_expert_ffn_noalloc", "moe_layer_workspace", "moe_layer", "moe_add_rms_norm", "moe_combine_norm",
    "moe_shared_ffn_workspace", "moe_shared_ffn", "moe_grouped_linear", "moe_grouped_dgrad", "moe_grouped_wgrad",
    "moe_q4_linear",
]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


class LayerDesc(ctypes.Structure):
    """moe_layer_desc (include/moe2bit.h)."""
    _fields_ = [
        ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("gate_up_fmt", ctypes.c_int32), ("down_fmt", ctypes.c_int32),
        ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
        ("codebook", ctypes.c_void_p),
        ("shared_inter", ctypes.c_int32),
        ("shared_gate", ctypes.c_void_p), ("shared_up", ctypes.c_void_p), ("shared_down", ctypes.c_void_p),
        ("path", ctypes.c_int32),
        ("precision", ctypes.c_int32),
    ]


class AdapterDesc(ctypes.Structure):
    """moe_adapter_desc (include/moe2bit.h)."""
    _fields_ = [
        ("n_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32),
        ("rank", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("gate_a", ctypes.c_void_p), ("gate_b", ctypes.c_void_p), ("up_a", ctypes.c_void_p), ("up_b", ctypes.c_void_p),
        ("down_a", ctypes.c_void_p), ("down_b", ctypes.c_void_p),
    ]


class GroupDesc(ctypes.Structure):
    """moe_group_desc (include/moe2bit.h)."""
    _fields_ = [
        ("n_groups", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("offsets", ctypes.c_void_p),
        ("in_index", ctypes.c_void_p), ("in_div", ctypes.c_int32), ("out_index", ctypes.c_void_p),
    ]


class Q4Desc(ctypes.Structure):
    """moe_q4_desc (include/moe2bit.h)."""
    _fields_ = [
        ("n_mats", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("group", ctypes.c_int32),
        ("scale_dt", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python bit_quantized_moe_permute_amd/build.py` "
                          f"(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_abi_version.argtypes = []
    L.moe_sync_debug.restype = ctypes.c_int
    L.moe_sync_debug.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_last_error.argtypes = []
    L.moe_weight_bytes.restype = sz
    L.moe_weight_bytes.argtypes = [i32, i64, i64, i64]
    L.moe_prepare_weights.restype = ctypes.c_int
    L.moe_prepare_weights.argtypes = [i32, i64, i64, i64, vp, vp, vp]
    L.moe_dequantize.restype = ctypes.c_int
    L.moe_dequantize.argtypes = [i32, vp, i64, i64, i64, i64, i64, vp, vp, vp]
    L.moe_route_workspace.restype = sz
    L.moe_route_workspace.argtypes = [i32, i32, i32]
    L.moe_route.restype = ctypes.c_int
    L.moe_route.argtypes = [vp, i32, i32, i32, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_ffn_workspace.restype = sz
    L.moe_expert_ffn_workspace.argtypes = [ctypes.POINTER(LayerDesc), i32]
    L.moe_expert_ffn.restype = ctypes.c_int
    L.moe_expert_ffn.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_gate_up.restype = ctypes.c_int
    L.moe_expert_gate_up.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_down.restype = ctypes.c_int
    L.moe_expert_down.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_combine.restype = ctypes.c_int
    L.moe_combine.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    L.moe_combine_steer.restype = ctypes.c_int
    L.moe_combine_steer.argtypes = [vp, vp, vp, i32, i32, i32, vp, ctypes.c_float, vp, vp]
    L.moe_expert_ffn_noalloc.restype = ctypes.c_int
    L.moe_expert_ffn_noalloc.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.moe_layer_workspace.restype = sz
    L.moe_layer_workspace.argtypes = [ctypes.POINTER(LayerDesc), i32]
    L.moe_layer.restype = ctypes.c_int
    L.moe_layer.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                            ctypes.c_float, vp, vp, sz, vp]
    L.moe_add_rms_norm.restype = ctypes.c_int
    L.moe_add_rms_norm.argtypes = [vp, i32, i32, i32, vp, vp, i32, vp, i32, ctypes.c_float, vp, i32, vp, vp]
    L.moe_combine_norm.restype = ctypes.c_int
    L.moe_combine_norm.argtypes = [vp, vp, vp, i32, i32, i32, vp, ctypes.c_float, vp, vp, i32, vp, i32,
                                   ctypes.c_float, vp, i32, vp, vp]
    L.moe_shared_ffn_workspace.restype = sz
    L.moe_shared_ffn_workspace.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(AdapterDesc), i32]
    L.moe_shared_ffn.restype = ctypes.c_int
    L.moe_shared_ffn.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(AdapterDesc), vp, i32, i32, vp, vp, i32, vp,
                                 sz, vp]
    gd = ctypes.POINTER(GroupDesc)
    L.moe_grouped_linear.restype = ctypes.c_int
    L.moe_grouped_linear.argtypes = [gd, vp, i32, vp, i32, i32, i32, vp, i32, i32, vp]
    L.moe_grouped_dgrad.restype = ctypes.c_int
    L.moe_grouped_dgrad.argtypes = [gd, vp, i32, vp, i32, i32, vp, i32, i32, vp]
    L.moe_grouped_wgrad.restype = ctypes.c_int
    L.moe_grouped_wgrad.argtypes = [gd, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp]
    L.moe_q4_linear.restype = ctypes.c_int
    L.moe_q4_linear.argtypes = [gd, ctypes.POINTER(Q4Desc), vp, i32, i32, vp, i32, i32, vp]
    L.moe_probe_stream_read.restype = ctypes.c_int
    L.moe_probe_stream_read.argtypes = [vp, sz, vp, i32, vp]
    if L.moe_abi_version() != ABI_VERSION:
        raise ImportError(f"libmoe2bit ABI {L.moe_abi_version()} != binding ABI {ABI_VERSION}")
    return L


lib = _load()


def _check(st: int):
    if st != MOE_OK:
        raise MoeError(st, lib.moe_last_error().decode())


def _ptr(t, dtype=None):
    """Device pointer of a contiguous GPU tensor (None passes through); dtype, when given, is checked."""
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError("expected a GPU tensor (the library takes device pointers)")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _i32(t):
    import torch
    return _ptr(t, torch.int32)


def _f32(t):
    import torch
    return _ptr(t, torch.float32)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, n: int, what: str):
    """Host-side size check before a device pointer is handed to the library: the kernels index t up to n
    elements (None passes)."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{what}: {t.numel()} elements, the call needs {n}")


def _need_bytes(t, n: int, what: str):
    if t is not None and t.numel() * t.element_size() < n:
        raise ValueError(f"{what}: {t.numel() * t.element_size()} bytes, the call needs {n}")


def _rows(x, hidden: int | None = None):
    """(T, H) of a [T][H] activation tensor."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"activations must be [tokens][hidden], got shape {tuple(shape)}")
    if hidden is not None and shape[1] != hidden:
        raise ValueError(f"activations have {shape[1]} columns, the layer has hidden {hidden}")
    return shape


def _dt(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return DT_BF16
    if t.dtype == torch.float32:
        return DT_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------------------
# C-ABI calls (same names)
# ----------------------------------------------------------------------------
def moe_abi_version() -> int:
    return lib.moe_abi_version()


def moe_sync_debug() -> bool:
    return bool(lib.moe_sync_debug())


def moe_last_error() -> str:
    return lib.moe_last_error().decode()


def moe_weight_bytes(fmt: int, n_mats: int, rows: int, cols: int) -> int:
    return lib.moe_weight_bytes(fmt, n_mats, rows, cols)


def moe_prepare_weights(fmt, n_mats, rows, cols, canonical, prepared, stream=None):
    nb = moe_weight_bytes(fmt, n_mats, rows, cols)
    _need_bytes(canonical, nb, "canonical")
    _need_bytes(prepared, nb, "prepared")
    _check(lib.moe_prepare_weights(fmt, n_mats, rows, cols, _ptr(canonical), _ptr(prepared), _stream(stream)))


def moe_dequantize(fmt, prepared, n_mats, rows, cols, mat_begin, mat_count, codebook, out, stream=None):
    _need_bytes(prepared, moe_weight_bytes(fmt, n_mats, rows, cols), "prepared")
    _need(out, max(mat_count, 0) * rows * cols, "out")
    if fmt == FMT_IQ2X:
        _need_bytes(codebook, 256 * 8, "codebook")
    _check(lib.moe_dequantize(fmt, _ptr(prepared), n_mats, rows, cols, mat_begin, mat_count, _ptr(codebook),
                              _f32(out), _stream(stream)))


def moe_route_workspace(n_tokens: int, n_experts: int, top_k: int) -> int:
    return lib.moe_route_workspace(n_tokens, n_experts, top_k)


def moe_route(x, w_router, n_experts, top_k, topk_idx, topk_w, expert_offsets, perm, active, ws, bias=None,
              logits=None, stream=None):
    T, H = _rows(x)
    if w_router.dim() != 2 or tuple(w_router.shape) != (n_experts, H):
        raise ValueError(f"w_router must be [{n_experts}][{H}], got shape {tuple(w_router.shape)}")
    _need(topk_idx, T * top_k, "topk_idx")
    _need(topk_w, T * top_k, "topk_w")
    _need(expert_offsets, n_experts + 1, "expert_offsets")
    _need(perm, T * top_k, "perm")
    _need(active, n_experts + 1, "active")
    _need(bias, n_experts, "bias")
    _need(logits, T * n_experts, "logits")
    _check(lib.moe_route(_ptr(x), _dt(x), T, H, _ptr(w_router), _dt(w_router), n_experts, _f32(bias), top_k,
                         _i32(topk_idx), _f32(topk_w), _f32(logits), _i32(expert_offsets), _i32(perm), _i32(active),
                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_ffn_workspace(desc: LayerDesc, n_tokens: int) -> int:
    return lib.moe_expert_ffn_workspace(ctypes.byref(desc), n_tokens)


def _routing_sizes(desc: LayerDesc, x, topk_idx, expert_offsets, perm, active):
    T, _ = _rows(x, desc.hidden)
    _need(topk_idx, T * desc.top_k, "topk_idx")
    _need(expert_offsets, desc.n_experts + 1, "expert_offsets")
    _need(perm, T * desc.top_k, "perm")
    _need(active, desc.n_experts + 1, "active")
    return T


def _output_sizes(desc: LayerDesc, T: int, slot_out, shared_out):
    _need(slot_out, T * desc.top_k * desc.hidden, "slot_out")
    _need(shared_out, T * desc.hidden, "shared_out")


def moe_expert_ffn(desc: LayerDesc, x, topk_idx, expert_offsets, perm, active, slot_out, shared_out, ws, stream=None):
    T = _routing_sizes(desc, x, topk_idx, expert_offsets, perm, active)
    _output_sizes(desc, T, slot_out, shared_out)
    _check(lib.moe_expert_ffn(ctypes.byref(desc), _ptr(x), _dt(x), T, _i32(topk_idx), _i32(expert_offsets),
                              _i32(perm), _i32(active), _f32(slot_out), _f32(shared_out), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_ffn_noalloc(desc: LayerDesc, x, topk_idx, expert_offsets, perm, active, slot_out, shared_out,
                           stream=None):
    """moe_expert_ffn with the library's static device scratch instead of a workspace (no allocation)."""
    T = _routing_sizes(desc, x, topk_idx, expert_offsets, perm, active)
    _output_sizes(desc, T, slot_out, shared_out)
    _check(lib.moe_expert_ffn_noalloc(ctypes.byref(desc), _ptr(x), _dt(x), T, _i32(topk_idx), _i32(expert_offsets),
                                      _i32(perm), _i32(active), _f32(slot_out), _f32(shared_out), _stream(stream)))


def moe_expert_gate_up(desc: LayerDesc, x, topk_idx, expert_offsets, perm, active, ws, stream=None):
    _routing_sizes(desc, x, topk_idx, expert_offsets, perm, active)
    _check(lib.moe_expert_gate_up(ctypes.byref(desc), _ptr(x), _dt(x), x.shape[0], _i32(topk_idx),
                                  _i32(expert_offsets), _i32(perm), _i32(active), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_down(desc: LayerDesc, x, topk_idx, expert_offsets, perm, active, slot_out, shared_out, ws, stream=None):
    T = _routing_sizes(desc, x, topk_idx, expert_offsets, perm, active)
    _output_sizes(desc, T, slot_out, shared_out)
    _check(lib.moe_expert_down(ctypes.byref(desc), _ptr(x), _dt(x), x.shape[0], _i32(topk_idx),
                               _i32(expert_offsets), _i32(perm), _i32(active), _f32(slot_out), _f32(shared_out),
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def _combine_sizes(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, y):
    _need(slot_out, n_tokens * top_k * hidden, "slot_out")
    _need(topk_w, n_tokens * top_k, "topk_w")
    _need(shared_out, n_tokens * hidden, "shared_out")
    _need(y, n_tokens * hidden, "y")


def moe_combine(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, y, stream=None):
    _combine_sizes(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, y)
    _check(lib.moe_combine(_f32(slot_out), _f32(topk_w), _f32(shared_out), n_tokens, top_k, hidden, _f32(y),
                           _stream(stream)))


def moe_combine_steer(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, steer_v, steer_f, y, stream=None):
    _combine_sizes(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, y)
    _need(steer_v, hidden, "steer_v")
    _check(lib.moe_combine_steer(_f32(slot_out), _f32(topk_w), _f32(shared_out), n_tokens, top_k, hidden,
                                 _f32(steer_v), float(steer_f), _f32(y), _stream(stream)))


def moe_layer_workspace(desc: LayerDesc, n_tokens: int) -> int:
    return lib.moe_layer_workspace(ctypes.byref(desc), n_tokens)


def moe_layer(desc: LayerDesc, x, w_router, topk_idx, topk_w, expert_offsets, perm, active, slot_out, shared_out, y,
              ws, bias=None, logits=None, steer_v=None, steer_f=0.0, stream=None):
    """route -> expert FFN -> combine (+ steering when steer_v is given) in one C-ABI call."""
    T = _routing_sizes(desc, x, topk_idx, expert_offsets, perm, active)
    if w_router.dim() != 2 or tuple(w_router.shape) != (desc.n_experts, desc.hidden):
        raise ValueError(f"w_router must be [{desc.n_experts}][{desc.hidden}], got shape {tuple(w_router.shape)}")
    _output_sizes(desc, T, slot_out, shared_out)
    _need(topk_w, T * desc.top_k, "topk_w")
    _need(bias, desc.n_experts, "bias")
    _need(logits, T * desc.n_experts, "logits")
    _need(steer_v, desc.hidden, "steer_v")
    _need(y, T * desc.hidden, "y")
    _check(lib.moe_layer(ctypes.byref(desc), _ptr(x), _dt(x), T, _ptr(w_router), _dt(w_router), _f32(bias),
                         _i32(topk_idx), _f32(topk_w), _f32(logits), _i32(expert_offsets), _i32(perm), _i32(active),
                         _f32(slot_out), _f32(shared_out), _f32(steer_v), float(steer_f), _f32(y), _ptr(ws),
                         ws.numel() * ws.element_size(), _stream(stream)))


def _addrs(dev, *tensors):
    """Addresses (ints) of contiguous tensors on GPU `dev`; None passes."""
    if dev < 0:
        raise TypeError("expected a GPU tensor (the library takes device pointers)")
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != dev:
            if not t.is_cuda:
                raise TypeError("expected a GPU tensor (the library takes device pointers)")
            raise ValueError(f"tensors on devices {dev} and {t.get_device()}")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        out.append(t.data_ptr())
    return out


def _stream_on(stream, dev):
    """The given stream, or torch's current one on GPU `dev`, which has to be the current device (the library
    launches there)."""
    now = torch._C._cuda_getDevice()
    if dev != now:
        raise ValueError(f"tensors on device {dev}, the current device is {now}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream


def _type(t, what):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    return dt


def _norm_output(dev, T, H, residual, residual_out, weight, y, y_scale):
    """Shape, type and device checks of what the norm calls share; their arguments from the residual on: addresses and types
    of residual, weight and output.  (A one-row call is bound by these checks: each tensor is asked once for what is needed.)"""
    n = T * H
    pr = po = ps = None
    res_dt = DT_F32
    if residual is not None and residual_out is not None:
        res_t = residual.dtype
        res_dt = _DTYPES.get(res_t)
        if res_dt is None:
            _type(residual, "residual")
        if residual_out is not residual:
            if residual_out.dtype != res_t:
                raise TypeError(f"residual_out: expected {res_t}, got {residual_out.dtype}")
            if residual_out.numel() < n:
                _need(residual_out, n, "residual_out")
            if not residual_out.is_contiguous() or residual_out.get_device() != dev:
                _addrs(dev, residual_out)
            po = residual_out.data_ptr()
        if residual.numel() < n:
            _need(residual, n, "residual")
        if not residual.is_contiguous() or residual.get_device() != dev:
            _addrs(dev, residual)
        pr = residual.data_ptr()
        if po is None:
            po = pr
    elif residual is not None or residual_out is not None:
        raise ValueError("residual_out must be given iff residual is")
    if weight.numel() < H or y.numel() < n:
        _need(weight, H, "weight")
        _need(y, n, "y")
    y_t = y.dtype
    w_dt, y_dt = _DTYPES.get(weight.dtype), _DTYPES.get(y_t)
    if w_dt is None:
        _type(weight, "weight")
    if y_scale is None:
        if y_t == torch.float8_e4m3fn:
            raise ValueError("y_scale is given iff y is float8_e4m3fn")
        if y_dt is None:
            _type(y, "y")
    elif y_t != torch.float8_e4m3fn:
        raise ValueError("y_scale is given iff y is float8_e4m3fn")
    elif y_scale.dtype == torch.float32:
        _need(y_scale, T, "y_scale")
        y_dt = DT_E4M3_ROW
    elif y_scale.dtype in (torch.float8_e8m0fnu, torch.uint8):
        _need(y_scale, T * ((H + 31) // 32), "y_scale")
        y_dt = DT_E4M3_BLOCK
    else:
        raise TypeError(f"y_scale: expected float32 (row scales), float8_e8m0fnu or uint8 (block scales), got "
                        f"{y_scale.dtype}")
    if not (weight.is_contiguous() and y.is_contiguous() and weight.get_device() == dev and y.get_device() == dev):
        _addrs(dev, weight, y)
    if y_scale is not None:
        ps, = _addrs(dev, y_scale)
    return pr, po, res_dt, weight.data_ptr(), w_dt, y.data_ptr(), y_dt, ps


def moe_add_rms_norm(x, residual, residual_out, weight, eps, y, y_scale=None, stream=None):
    """residual_out = x + residual; y = rms_norm(residual_out) * weight.  y float32, bfloat16, or float8_e4m3fn with
    y_scale float8_e8m0fnu / uint8 [T][ceil(H/32)] (block scales) or float32 [T] (row scales); residual and
    residual_out may be None together, or the same tensor."""
    T, H = _rows(x)
    dev = x.get_device()
    pr, po, res_dt, pw, w_dt, py, y_dt, ps = _norm_output(dev, T, H, residual, residual_out, weight, y, y_scale)
    x_dt = _type(x, "x")
    if dev < 0 or not x.is_contiguous():
        _addrs(dev, x)
    st = lib.moe_add_rms_norm(x.data_ptr(), x_dt, T, H, pr, po, res_dt, pw, w_dt, eps, py, y_dt, ps, _stream_on(stream, dev))
    if st:
        _check(st)


def moe_combine_norm(slot_out, topk_w, shared_out, residual, residual_out, weight, eps, y, y_scale=None, steer_v=None,
                     steer_f=0.0, stream=None):
    """moe_add_rms_norm of the combine's result (steered when steer_v is given): slot_out [T*k][H], topk_w [T][k]."""
    (T, k), H = _rows(topk_w), _rows(slot_out)[1]
    if slot_out.numel() != T * k * H:
        raise ValueError(f"slot_out must be [T*k][H] and topk_w [T][k], got {tuple(slot_out.shape)} and "
                         f"{tuple(topk_w.shape)}")
    f32 = torch.float32
    dev, psh, pv = slot_out.get_device(), None, None
    if slot_out.dtype != f32 or topk_w.dtype != f32:
        raise TypeError(f"slot_out and topk_w: expected torch.float32, got {slot_out.dtype} and {topk_w.dtype}")
    if shared_out is not None:
        if shared_out.dtype != f32:
            raise TypeError(f"shared_out: expected torch.float32, got {shared_out.dtype}")
        if shared_out.numel() < T * H:
            _need(shared_out, T * H, "shared_out")
        if not shared_out.is_contiguous() or shared_out.get_device() != dev:
            _addrs(dev, shared_out)
        psh = shared_out.data_ptr()
    if steer_v is not None:
        if steer_v.dtype != f32:
            raise TypeError(f"steer_v: expected torch.float32, got {steer_v.dtype}")
        _need(steer_v, H, "steer_v")
        pv, = _addrs(dev, steer_v)
    pr, po, res_dt, pw, w_dt, py, y_dt, ps = _norm_output(dev, T, H, residual, residual_out, weight, y, y_scale)
    if dev < 0 or not (slot_out.is_contiguous() and topk_w.is_contiguous() and topk_w.get_device() == dev):
        _addrs(dev, slot_out, topk_w)
    st = lib.moe_combine_norm(slot_out.data_ptr(), topk_w.data_ptr(), psh, T, k, H, pv, steer_f, pr, po, res_dt, pw, w_dt, eps,
                              py, y_dt, ps, _stream_on(stream, dev))
    if st:
        _check(st)


def moe_shared_ffn_workspace(desc: LayerDesc, n_tokens: int, adapters=None) -> int:
    """adapters: an AdapterPool, or None."""
    return lib.moe_shared_ffn_workspace(desc, None if adapters is None else adapters.desc, n_tokens)


def moe_shared_ffn(desc: LayerDesc, x, out, ws, adapters=None, token_adapter=None, stream=None):
    """The layer's shared expert on x [T][H] into out [T][H], token t through adapter token_adapter[t] of the
    AdapterPool `adapters` (an index outside the pool: none)."""
    T, H = _rows(x, desc.hidden)
    if out.numel() < T * H:
        _need(out, T * H, "out")
    dev, pool = x.get_device(), None
    if adapters is not None:
        if (adapters.hidden, adapters.inter) != (H, desc.shared_inter):
            raise ValueError(f"adapters are for hidden {adapters.hidden}, inter {adapters.inter}; the layer has "
                             f"{H}, {desc.shared_inter}")
        if adapters.device_index != dev and dev >= 0:
            raise ValueError(f"tensors on devices {dev} and {adapters.device_index}")
        if token_adapter is None or token_adapter.dtype != torch.int32:
            raise TypeError("token_adapter must be an int32 tensor")
        _need(token_adapter, T, "token_adapter")
        pool = adapters.desc
    x_dt, out_dt = _type(x, "x"), _type(out, "out")
    px, pi, po, pws = _addrs(dev, x, token_adapter, out, ws)
    st = lib.moe_shared_ffn(desc, pool, px, x_dt, T, pi, po, out_dt, pws, ws.numel() * ws.element_size(),
                            _stream_on(stream, dev))
    if st:
        _check(st)


_I32_MAX = 2**31 - 1


def _bf16_rows(t, what, cols):
    """Rows of a [rows][cols] bf16 tensor (those that an int32 can name)."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError(f"{what} must be [rows][{cols}], got shape {tuple(shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: expected torch.bfloat16, got {t.dtype}")
    return min(shape[0], _I32_MAX)


def _out_rows(t, what, cols):
    """Rows (those that an int32 can name) and type of a [rows][cols] output."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError(f"{what} must be [rows][{cols}], got shape {tuple(shape)}")
    return min(shape[0], _I32_MAX), _type(t, what)


def _stack(groups, w):
    """(n_out, n_in) of a bf16 [groups][n_out][n_in] stack."""
    shape = w.shape
    if len(shape) != 3 or shape[0] != groups.n:
        raise ValueError(f"weights must be [{groups.n}][n_out][n_in], got shape {tuple(shape)}")
    if w.dtype != torch.bfloat16:
        raise TypeError(f"weights: expected torch.bfloat16, got {w.dtype}")
    return shape[1], shape[2]


def _group_dev(groups, dev):
    if groups.device_index is not None and groups.device_index != dev and dev >= 0:
        raise ValueError(f"tensors on devices {dev} and {groups.device_index}")


def moe_grouped_linear(groups, x, w, out, act=ACT_NONE, stream=None):
    """out[o] = W_g x[r] for the rows of every group of `groups` (a RowGroups); x [rows][n_in] bf16, w
    [groups][n_out][n_in] bf16, out [rows][n_out] float32 or bfloat16.  ACT_SWIGLU: w [groups][2 n_out][n_in], gate rows
    then up rows, out = silu(gate) * up."""
    N, K = _stack(groups, w)
    if act == ACT_SWIGLU:
        if N % 2:
            raise ValueError(f"weights of a SwiGLU must have an even number of rows, got {N}")
        N //= 2
    x_rows = _bf16_rows(x, "x", K)
    out_rows, out_dt = _out_rows(out, "out", N)
    dev = x.get_device()
    _group_dev(groups, dev)
    px, pw, po = _addrs(dev, x, w, out)
    st = lib.moe_grouped_linear(groups.desc, px, x_rows, pw, N, K, act, po, out_dt, out_rows, _stream_on(stream, dev))
    if st:
        _check(st)


def moe_grouped_dgrad(groups, dy, w, dx, stream=None):
    """The gradient of moe_grouped_linear (without activation) with respect to its input: dx[in_index[i], or i] =
    W_g^T dy[o]; dy [rows][n_out] bf16, dx [rows][n_in] float32 or bfloat16."""
    N, K = _stack(groups, w)
    dy_rows = _bf16_rows(dy, "dy", N)
    dx_rows, dx_dt = _out_rows(dx, "dx", K)
    dev = dy.get_device()
    _group_dev(groups, dev)
    py, pw, po = _addrs(dev, dy, w, dx)
    st = lib.moe_grouped_dgrad(groups.desc, py, dy_rows, pw, N, K, po, dx_dt, dx_rows, _stream_on(stream, dev))
    if st:
        _check(st)


def moe_grouped_wgrad(groups, x, dy, dw, accumulate=False, stream=None):
    """The gradient of moe_grouped_linear (without activation) with respect to its weights: dw[g] (+)= the sum of
    dy[o] x[r]^T over the rows of group g; x [rows][n_in] and dy [rows][n_out] bf16, dw [groups][n_out][n_in] float32 or
    bfloat16."""
    shape = dw.shape
    if len(shape) != 3 or shape[0] != groups.n:
        raise ValueError(f"dw must be [{groups.n}][n_out][n_in], got shape {tuple(shape)}")
    N, K = shape[1], shape[2]
    x_rows, dy_rows, dw_dt = _bf16_rows(x, "x", K), _bf16_rows(dy, "dy", N), _type(dw, "dw")
    dev = x.get_device()
    _group_dev(groups, dev)
    px, py, po = _addrs(dev, x, dy, dw)
    st = lib.moe_grouped_wgrad(groups.desc, px, x_rows, py, dy_rows, N, K, bool(accumulate), po, dw_dt,
                               _stream_on(stream, dev))
    if st:
        _check(st)


def moe_q4_linear(groups, weights, x, out, act=ACT_NONE, stream=None):
    """moe_grouped_linear with 4-bit weights (a Q4Weights with a matrix for every group of `groups`)."""
    N = weights.rows
    if act == ACT_SWIGLU:
        if N % 2:
            raise ValueError(f"weights of a SwiGLU must have an even number of rows, got {N}")
        N //= 2
    x_rows = _bf16_rows(x, "x", weights.cols)
    out_rows, out_dt = _out_rows(out, "out", N)
    dev = x.get_device()
    _group_dev(groups, dev)
    if weights.device_index != dev and dev >= 0:
        raise ValueError(f"tensors on devices {dev} and {weights.device_index}")
    px, po = _addrs(dev, x, out)
    st = lib.moe_q4_linear(groups.desc, weights.desc, px, x_rows, act, po, out_dt, out_rows, _stream_on(stream, dev))
    if st:
        _check(st)


def moe_probe_stream_read(buf, nbytes, sink, n_blocks, stream=None):
    """Measurement helper: one streaming read of buf's first nbytes bytes (sink: n_blocks uint32 words)."""
    _need_bytes(buf, nbytes, "buf")
    _need_bytes(sink, 4 * n_blocks, "sink")
    _check(lib.moe_probe_stream_read(_ptr(buf), nbytes, _ptr(sink), n_blocks, _stream(stream)))


import torch  # noqa: E402  (after the library: it fails first where it is missing)

_DTYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}

from .layer import AdapterPool, DeviceLayer, LayerBuffers, Q4Weights, RowGroups  # noqa: E402  (needs `lib` loaded)
