"""Python binding of librowops.so (argument marshalling only).

Each function has the name of the C entry point it calls and does no
arithmetic of its own: it checks shapes, takes device pointers, the row stride
and the current CUDA stream from torch tensors, calls the C ABI through
ctypes and raises :class:`RowopsError` on a non-OK status. PyTorch only
supplies device memory and streams. There is no CPU fallback: if the library
is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB as _LIB_PATH

__all__ = [
    "RowopsError",
    "library",
    "library_path",
    "rowops_softmax",
    "rowops_softmax_causal",
    "rowops_row_sum",
    "rowops_row_max",
    "rowops_online_softmax",
    "rowops_online_softmax_workspace_bytes",
    "rowops_online_softmax_status",
    "rowops_online_softmax_noalloc",
    "rowops_device_status",
    "rowops_layernorm_gelu",
    "rowops_layernorm_gelu_erf",
    "rowops_layernorm_gelu_backward",
    "rowops_layernorm_gelu_backward_workspace_bytes",
    "rowops_gelu",
    "rowops_bias_residual_gelu",
    "rowops_rmsnorm",
    "rowops_fused_residual_rmsnorm",
    "rowops_groupnorm_act",
    "rowops_groupnorm_act_workspace_bytes",
    "rowops_groupnorm_act_backward",
    "rowops_groupnorm_act_backward_workspace_bytes",
    "rowops_bias_dropout_residual",
    "rowops_bias_dropout_residual_backward",
    "rowops_bias_dropout_residual_backward_workspace_bytes",
    "rowops_router_balance_loss",
    "rowops_router_balance_loss_workspace_bytes",
    "rowops_router_balance_loss_backward",
    "rowops_rmsnorm_quant",
    "rowops_paged_attention",
    "rowops_paged_attention_workspace_bytes",
    "rowops_sample",
    "rowops_status_string",
    "rowops_reload_tuning",
    "ROWOPS_F32",
    "ROWOPS_BF16",
    "STATUS",
]

ROWOPS_F32 = 0
ROWOPS_BF16 = 1
STATUS = {
    0: "ROWOPS_OK",
    1: "ROWOPS_ERR_INVALID_VALUE",
    2: "ROWOPS_ERR_UNSUPPORTED",
    3: "ROWOPS_ERR_WORKSPACE",
    4: "ROWOPS_ERR_CUDA",
    5: "ROWOPS_ERR_TIMEOUT",
}

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class RowopsError(RuntimeError):
    """A rowops entry point returned a status other than ROWOPS_OK."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load librowops.so (built in-tree by ``row_wise_reduction_gb300.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m row_wise_reduction_gb300.build` "
                "(there is no fallback implementation)"
            )
        L = ctypes.CDLL(_LIB_PATH)
        L.rowops_status_string.restype = ctypes.c_char_p
        L.rowops_status_string.argtypes = [ctypes.c_int]
        L.rowops_reload_tuning.restype = None
        L.rowops_reload_tuning.argtypes = []
        L.rowops_softmax.restype = ctypes.c_int
        L.rowops_softmax.argtypes = [_vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp]
        L.rowops_online_softmax_workspace_bytes.restype = ctypes.c_size_t
        L.rowops_online_softmax_workspace_bytes.argtypes = [_i64, _i64, ctypes.c_int]
        L.rowops_online_softmax.restype = ctypes.c_int
        L.rowops_online_softmax.argtypes = [_vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp, ctypes.c_size_t,
                                            _i64, _vp]
        L.rowops_online_softmax_status.restype = ctypes.c_int
        L.rowops_online_softmax_status.argtypes = [_vp, _vp]
        L.rowops_device_status.restype = ctypes.c_int
        L.rowops_device_status.argtypes = [_vp]
        L.rowops_online_softmax_noalloc.restype = ctypes.c_int
        L.rowops_online_softmax_noalloc.argtypes = [_vp, _vp, _i64, _i64, _i64, ctypes.c_int, _i64, _vp]
        L.rowops_layernorm_gelu.restype = ctypes.c_int
        L.rowops_layernorm_gelu.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_float, _i64, _i64, _i64,
                                            ctypes.c_int, _vp]
        for name in ("rowops_row_sum", "rowops_row_max"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [_vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp]
        L.rowops_softmax_causal.restype = ctypes.c_int
        L.rowops_softmax_causal.argtypes = [_vp, _vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _vp]
        L.rowops_layernorm_gelu_erf.restype = ctypes.c_int
        L.rowops_layernorm_gelu_erf.argtypes = L.rowops_layernorm_gelu.argtypes
        L.rowops_gelu.restype = ctypes.c_int
        L.rowops_gelu.argtypes = [_vp, _vp, _i64, ctypes.c_int, ctypes.c_int, _vp]
        L.rowops_rmsnorm.restype = ctypes.c_int
        L.rowops_rmsnorm.argtypes = [_vp, _vp, _vp, ctypes.c_float, _i64, _i64, _i64, ctypes.c_int, _vp]
        L.rowops_fused_residual_rmsnorm.restype = ctypes.c_int
        L.rowops_fused_residual_rmsnorm.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_float, _i64, _i64, _i64,
                                                    ctypes.c_int, _vp]
        L.rowops_bias_residual_gelu.restype = ctypes.c_int
        L.rowops_bias_residual_gelu.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                                _vp]
        L.rowops_layernorm_gelu_backward_workspace_bytes.restype = ctypes.c_size_t
        L.rowops_layernorm_gelu_backward_workspace_bytes.argtypes = [_i64, _i64, ctypes.c_int]
        L.rowops_layernorm_gelu_backward.restype = ctypes.c_int
        L.rowops_layernorm_gelu_backward.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _i64,
                                                     _i64, _i64, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        u64, size, i32, f32 = ctypes.c_uint64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        for name, res, args in (
            ("groupnorm_act_workspace_bytes", size, [_i64] * 4 + [i32]),
            ("groupnorm_act", i32, [_vp] * 4 + [f32] + [_i64] * 5 + [i32, _vp, i32, _vp, size, _vp]),
            ("groupnorm_act_backward_workspace_bytes", size, [_i64] * 4 + [i32]),
            ("groupnorm_act_backward", i32, [_vp] * 8 + [_i64] * 5 + [i32, i32, _vp, size, _vp]),
            ("bias_dropout_residual", i32, [_vp] * 4 + [f32, u64, u64, _vp] + [_i64] * 3 + [i32, _vp]),
            ("bias_dropout_residual_backward_workspace_bytes", size, [_i64] * 2 + [i32]),
            ("bias_dropout_residual_backward", i32,
             [_vp] * 3 + [f32, u64, u64, _vp] + [_i64] * 3 + [i32, _vp, size, _vp]),
            ("router_balance_loss_workspace_bytes", size, [_i64] * 2 + [i32]),
            ("router_balance_loss", i32,
             [_vp, _vp, i32, _vp, f32, _vp, _vp] + [_i64] * 4 + [i32, _vp, size, _vp]),
            ("router_balance_loss_backward", i32, [_vp] * 4 + [f32, _vp] + [_i64] * 4 + [i32, _vp]),
            ("rmsnorm_quant", i32, [_vp] * 6 + [f32] + [_i64] * 5 + [i32, _vp]),
            ("paged_attention_workspace_bytes", size, [_i64] * 7 + [i32]),
            ("paged_attention", i32, [_vp] * 7 + [f32] + [_i64] * 14 + [i32, _vp, size, _vp]),
            ("sample", i32, [_vp] * 3 + [f32, _vp, ctypes.c_int32, _vp, f32, _vp, f32] + [_vp] * 2 + [_i64] * 3
             + [i32, _vp]),
        ):
            f = getattr(L, "rowops_" + name)
            f.restype, f.argtypes = res, args
        _bind_calls(L)  # before _lib: a thread that sees _lib set finds _calls set too
        _lib = L
    return _lib


_OPERATORS = (
    "groupnorm_act_workspace_bytes",
    "groupnorm_act",
    "groupnorm_act_backward_workspace_bytes",
    "groupnorm_act_backward",
    "bias_dropout_residual",
    "bias_dropout_residual_backward_workspace_bytes",
    "bias_dropout_residual_backward",
    "router_balance_loss",
    "router_balance_loss_backward",
    "router_balance_loss_workspace_bytes",
    "rmsnorm_quant",
    "paged_attention_workspace_bytes",
    "paged_attention",
    "sample",
)


class _Calls:
    """The entry points whose small calls are bound by host time: through the
    CPython call module ``_rowops_call`` where it was built (about 0.1 us of
    marshalling per call), else through ctypes (about 2 us)."""

    __slots__ = ("softmax", "layernorm_gelu", "layernorm_gelu_erf", "module") + _OPERATORS


_calls: Optional[_Calls] = None


def _bind_calls(L: ctypes.CDLL) -> None:
    global _calls
    c = _Calls()
    try:
        from . import _rowops_call as fast
    except ImportError:
        fast = None
    if fast is not None:
        def addr(f):
            return ctypes.cast(f, ctypes.c_void_p).value

        fast.bind(addr(L.rowops_softmax), addr(L.rowops_layernorm_gelu), addr(L.rowops_layernorm_gelu_erf))
        c.softmax, c.layernorm_gelu, c.layernorm_gelu_erf = fast.softmax, fast.layernorm_gelu, fast.layernorm_gelu_erf
    else:
        c.softmax, c.layernorm_gelu, c.layernorm_gelu_erf = (L.rowops_softmax, L.rowops_layernorm_gelu,
                                                              L.rowops_layernorm_gelu_erf)
    if fast is not None:
        fast.bind_operators(*(addr(getattr(L, "rowops_" + n)) for n in _OPERATORS))
    for n in _OPERATORS:
        setattr(c, n, getattr(L, "rowops_" + n) if fast is None else getattr(fast, n))
    c.module = fast
    _calls = c


def _hot_calls() -> _Calls:
    library()
    return _calls


def rowops_status_string(status: int) -> str:
    return library().rowops_status_string(int(status)).decode()


def rowops_reload_tuning() -> None:
    """Make the library read the ROWOPS_* knobs from the environment again
    (it reads them once, at its first call, otherwise)."""
    library().rowops_reload_tuning()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return ROWOPS_F32
    if t.dtype == torch.bfloat16:
        return ROWOPS_BF16
    raise TypeError(f"rowops supports float32 and bfloat16, not {t.dtype}")


def _rows(t: torch.Tensor, name: str):
    """(M, N, ld) of a 2-D CUDA tensor with unit column stride. (Each tensor
    property is read once: at the small, launch-bound sizes the binding's own
    checks are a visible share of a call.)"""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    sh = t.shape
    if len(sh) != 2:
        raise ValueError(f"{name} must be 2-D (M, N)")
    M, N = sh
    st = t.stride()
    if N > 0 and st[1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    return M, N, (st[0] if M > 1 else max(N, st[0]))


def _out_like(x: torch.Tensor, y: Optional[torch.Tensor]) -> torch.Tensor:
    if y is None:
        return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
    if y.dtype is not x.dtype or y.get_device() != x.get_device() or y.shape != x.shape:
        raise ValueError("y must match x in shape, dtype and device")
    M, N = y.shape
    if y.stride() != x.stride() and (M > 1 or (M == 1 and N > 1 and y.stride(1) != 1)):
        raise ValueError("x and y must share the row stride")
    return y


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> int:
    if stream is None:
        # the raw handle of the current device's current stream (the cheap
        # form of torch.cuda.current_stream().cuda_stream; the tensors passed
        # in are CUDA tensors, so CUDA is initialised already)
        return _current_raw_stream(_current_device() if device is None else device)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_DTYPE_CODES = {torch.float32: ROWOPS_F32, torch.bfloat16: ROWOPS_BF16}


def _xy(x: torch.Tensor, y: Optional[torch.Tensor]):
    """_rows(x) and _out_like(x, y) in one pass over the tensors' properties,
    for the entry points whose small calls are bound by host time: returns
    (M, N, ld, y, dtype code, device index)."""
    sh = x.shape
    if len(sh) != 2:
        raise ValueError("x must be 2-D (M, N)")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a CUDA tensor")
    M, N = sh
    st = x.stride()
    if N > 0 and st[1] != 1:
        raise ValueError("x must have unit column stride")
    dt = x.dtype
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"rowops supports float32 and bfloat16, not {dt}")
    if y is None:
        y = torch.empty_strided(sh, st, dtype=dt, device=x.device)
    else:
        if y.dtype is not dt or y.get_device() != dev or y.shape != sh:
            raise ValueError("y must match x in shape, dtype and device")
        if y.stride() != st and (M > 1 or (M == 1 and N > 1 and y.stride(1) != 1)):
            raise ValueError("x and y must share the row stride")
    return M, N, (st[0] if M > 1 else max(N, st[0])), y, code, dev


def _check(fn: str, status: int):
    if status != 0:
        raise RowopsError(fn, status)


def rowops_softmax(x: torch.Tensor, y: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """Stable softmax of every row of ``x`` (M, N) into ``y`` (may be ``x``)."""
    M, N, ld, y, code, dev = _xy(x, y)
    st = (_calls or _hot_calls()).softmax(x.data_ptr(), y.data_ptr(), M, N, ld, code,
                                          _current_raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RowopsError("rowops_softmax", st)
    return y


def rowops_online_softmax_workspace_bytes(M: int, N: int, dtype: torch.dtype) -> int:
    code = ROWOPS_F32 if dtype == torch.float32 else ROWOPS_BF16 if dtype == torch.bfloat16 else -1
    return int(library().rowops_online_softmax_workspace_bytes(int(M), int(N), code))


def rowops_online_softmax(
    x: torch.Tensor,
    y: Optional[torch.Tensor] = None,
    *,
    workspace: Optional[torch.Tensor] = None,
    chunk: int = 0,
    stream=None,
) -> torch.Tensor:
    """Split-row online softmax of every row of ``x``.

    ``workspace``: a CUDA uint8 tensor of at least
    ``rowops_online_softmax_workspace_bytes(M, N, dtype)`` bytes; allocated
    here when omitted. ``chunk``: columns per CTA chunk (0 = automatic).
    """
    M, N, ld = _rows(x, "x")
    y = _out_like(x, y)
    need = rowops_online_softmax_workspace_bytes(M, N, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    st = library().rowops_online_softmax(x.data_ptr(), y.data_ptr(), M, N, ld, _dtype_code(x),
                                         workspace.data_ptr(), nbytes, int(chunk), _stream(stream))
    _check("rowops_online_softmax", st)
    return y


def rowops_online_softmax_status(workspace: torch.Tensor, *, stream=None) -> int:
    """Synchronise the stream and return the device-side status of the last
    rowops_online_softmax call on ``workspace`` (0 = ROWOPS_OK)."""
    return int(library().rowops_online_softmax_status(workspace.data_ptr(), _stream(stream)))


def rowops_device_status(*, stream=None) -> int:
    """Synchronise the stream, then read and clear the library's device error
    word on the current device (0 = ROWOPS_OK, 5 = a bounded device-side wait
    gave up)."""
    return int(library().rowops_device_status(_stream(stream)))


def rowops_online_softmax_noalloc(
    x: torch.Tensor, y: Optional[torch.Tensor] = None, *, chunk: int = 0, stream=None
) -> torch.Tensor:
    """rowops_online_softmax without a workspace, for callers that cannot
    allocate device memory: the partials live in the library's own 1 MiB
    device array (M * ceil(N / chunk) <= 131040). Calls that could overlap on
    the GPU share that array and must be ordered."""
    M, N, ld = _rows(x, "x")
    y = _out_like(x, y)
    st = library().rowops_online_softmax_noalloc(x.data_ptr(), y.data_ptr(), M, N, ld, _dtype_code(x), int(chunk),
                                                 _stream(stream))
    _check("rowops_online_softmax_noalloc", st)
    return y


def rowops_layernorm_gelu(
    x: torch.Tensor,
    w: Optional[torch.Tensor] = None,
    b: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    y: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """Fused LayerNorm -> affine -> tanh-GELU of every row of ``x``."""
    M, N, ld, y, code, dev = _xy(x, y)
    st = (_calls or _hot_calls()).layernorm_gelu(
        x.data_ptr(), y.data_ptr(), _affine(w, x, N, dev, "w"), _affine(b, x, N, dev, "b"), float(eps), M, N, ld,
        code, _current_raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RowopsError("rowops_layernorm_gelu", st)
    return y


def rowops_layernorm_gelu_erf(
    x: torch.Tensor,
    w: Optional[torch.Tensor] = None,
    b: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    y: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """Fused LayerNorm -> affine -> exact (erf) GELU of every row of ``x``."""
    M, N, ld, y, code, dev = _xy(x, y)
    st = (_calls or _hot_calls()).layernorm_gelu_erf(
        x.data_ptr(), y.data_ptr(), _affine(w, x, N, dev, "w"), _affine(b, x, N, dev, "b"), float(eps), M, N, ld,
        code, _current_raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RowopsError("rowops_layernorm_gelu_erf", st)
    return y


def rowops_layernorm_gelu_backward_workspace_bytes(M: int, N: int, dtype: torch.dtype) -> int:
    code = ROWOPS_F32 if dtype == torch.float32 else ROWOPS_BF16 if dtype == torch.bfloat16 else -1
    return int(library().rowops_layernorm_gelu_backward_workspace_bytes(int(M), int(N), code))


def _grad_out(t: Optional[torch.Tensor], N: int, device, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(N, dtype=torch.float32, device=device)
    if t.dtype != torch.float32 or t.numel() != N or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of N entries")
    return t


def rowops_layernorm_gelu_backward(
    x: torch.Tensor,
    dy: torch.Tensor,
    w: Optional[torch.Tensor] = None,
    b: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    dx: Optional[torch.Tensor] = None,
    dw: Optional[torch.Tensor] = None,
    db: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
    *,
    stream=None,
):
    """Gradients of rowops_layernorm_gelu (tanh GELU) for the upstream gradient
    ``dy``: returns ``(dx, dw, db)``, dx in x's dtype and layout, dw and db
    float32 (N,). ``workspace``: a CUDA uint8 tensor of at least
    ``rowops_layernorm_gelu_backward_workspace_bytes(M, N, dtype)`` bytes,
    allocated per call when omitted."""
    M, N, ld = _rows(x, "x")
    _out_like(x, dy)  # same shape, dtype, device and row stride
    dx = _out_like(x, dx)
    pw, pb = _weight(w, x, N, "w"), _weight(b, x, N, "b")
    dw = _grad_out(dw, N, x.device, "dw")
    db = _grad_out(db, N, x.device, "db")
    need = rowops_layernorm_gelu_backward_workspace_bytes(M, N, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    st = library().rowops_layernorm_gelu_backward(
        x.data_ptr(), dy.data_ptr(), pw, pb, float(eps), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), M, N, ld,
        _dtype_code(x), workspace.data_ptr(), nbytes, _stream(stream))
    _check("rowops_layernorm_gelu_backward", st)
    return dx, dw, db


def rowops_bias_residual_gelu(
    x: torch.Tensor,
    residual: Optional[torch.Tensor] = None,
    bias: Optional[torch.Tensor] = None,
    y: Optional[torch.Tensor] = None,
    approximate: str = "none",
    *,
    stream=None,
) -> torch.Tensor:
    """y = GELU(x + bias + residual) for every row of ``x`` (bias per column;
    residual shaped and strided like x; either may be None); approximate
    "none" (exact, erf) or "tanh"."""
    if approximate not in ("none", "tanh"):
        raise ValueError('approximate must be "none" or "tanh"')
    M, N, ld = _rows(x, "x")
    if residual is not None:
        _out_like(x, residual)  # same shape, dtype, device and row stride
    y = _out_like(x, y)
    st = library().rowops_bias_residual_gelu(
        x.data_ptr(), residual.data_ptr() if residual is not None else None, _weight(bias, x, N, "bias"),
        y.data_ptr(), M, N, ld, 0 if approximate == "none" else 1, _dtype_code(x), _stream(stream))
    _check("rowops_bias_residual_gelu", st)
    return y


def _affine(v: Optional[torch.Tensor], x: torch.Tensor, N: int, dev: int, name: str):
    """Device pointer of an optional per-column vector (w, b) of x's dtype."""
    if v is None:
        return None
    if v.dtype is not x.dtype or v.get_device() != dev or v.numel() != N or not v.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of N entries with x's dtype")
    return v.data_ptr()


def _weight(w: Optional[torch.Tensor], x: torch.Tensor, N: int, name: str = "w"):
    if w is None:
        return None
    if w.dtype != x.dtype or w.device != x.device or w.numel() != N or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of N entries with x's dtype")
    return w.data_ptr()


def rowops_rmsnorm(
    x: torch.Tensor,
    w: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    y: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """RMSNorm of every row of ``x``: x * rsqrt(mean(x^2) + eps) * w."""
    M, N, ld = _rows(x, "x")
    y = _out_like(x, y)
    st = library().rowops_rmsnorm(x.data_ptr(), y.data_ptr(), _weight(w, x, N), float(eps), M, N, ld,
                                  _dtype_code(x), _stream(stream))
    _check("rowops_rmsnorm", st)
    return y


def rowops_fused_residual_rmsnorm(
    x: torch.Tensor,
    residual: torch.Tensor,
    w: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    y: Optional[torch.Tensor] = None,
    residual_out: Optional[torch.Tensor] = None,
    *,
    stream=None,
):
    """residual_out = x + residual and y = RMSNorm(residual_out) * w, in one
    pass; returns ``(y, residual_out)``. Outputs may be given (e.g.
    ``residual_out=residual`` to update the residual stream in place)."""
    M, N, ld = _rows(x, "x")
    _out_like(x, residual)  # same shape, dtype, device and row stride
    y = _out_like(x, y)
    residual_out = _out_like(x, residual_out)
    st = library().rowops_fused_residual_rmsnorm(
        x.data_ptr(), residual.data_ptr(), y.data_ptr(), residual_out.data_ptr(), _weight(w, x, N), float(eps),
        M, N, ld, _dtype_code(x), _stream(stream))
    _check("rowops_fused_residual_rmsnorm", st)
    return y, residual_out


def rowops_softmax_causal(
    x: torch.Tensor,
    period: Optional[int] = None,
    offset: int = 0,
    y: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """Causal softmax: row r keeps the columns c <= (r mod period) + offset
    (default period: N, the stacked square causal masks); masked columns are
    not read and come out 0."""
    M, N, ld = _rows(x, "x")
    y = _out_like(x, y)
    period = N if period is None else int(period)
    st = library().rowops_softmax_causal(x.data_ptr(), y.data_ptr(), M, N, ld, period, int(offset),
                                         _dtype_code(x), _stream(stream))
    _check("rowops_softmax_causal", st)
    return y


def _row_reduce(fn: str, x: torch.Tensor, out: Optional[torch.Tensor], stream) -> torch.Tensor:
    M, N, ld = _rows(x, "x")
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=x.device)
    elif out.dtype != torch.float32 or out.numel() != M or not out.is_contiguous() or out.device != x.device:
        raise ValueError("out must be a contiguous float32 CUDA tensor of M entries")
    st = getattr(library(), fn)(x.data_ptr(), out.data_ptr(), M, N, ld, _dtype_code(x), _stream(stream))
    _check(fn, st)
    return out


def rowops_row_sum(x: torch.Tensor, out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """Sum of every row of ``x`` as float32 (M,)."""
    return _row_reduce("rowops_row_sum", x, out, stream)


def rowops_row_max(x: torch.Tensor, out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """Maximum of every row of ``x`` as float32 (M,); NaN where a row holds a NaN."""
    return _row_reduce("rowops_row_max", x, out, stream)


def rowops_gelu(x: torch.Tensor, y: Optional[torch.Tensor] = None, approximate: str = "none", *,
                stream=None) -> torch.Tensor:
    """Elementwise GELU of a contiguous tensor: approximate "none" (exact, erf)
    or "tanh"."""
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    if approximate not in ("none", "tanh"):
        raise ValueError('approximate must be "none" or "tanh"')
    if y is None:
        y = torch.empty_like(x)
    elif y.shape != x.shape or y.dtype != x.dtype or y.device != x.device or not y.is_contiguous():
        raise ValueError("y must be a contiguous tensor matching x")
    st = library().rowops_gelu(x.data_ptr(), y.data_ptr(), x.numel(), 0 if approximate == "none" else 1,
                               _dtype_code(x), _stream(stream))
    _check("rowops_gelu", st)
    return y


# ---------------------------------------------------------------------------
# Training operators: group norm + activation, bias + dropout + residual, the
# router's balance loss. Their calls run on the device of their tensors, and
# what they allocate is allocated on the stream that they run on.
# ---------------------------------------------------------------------------
def _elsewhere(fn, stream, dev, *args, **kwargs):
    """``fn`` with the tensors' device and ``stream`` current."""
    if dev < 0:
        raise ValueError("the call's tensors must be CUDA tensors")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        elif stream.device.index != dev:
            raise ValueError("stream must belong to the device of the call's tensors")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)


def _scratch(workspace: Optional[torch.Tensor], need: int, dev: int):
    """(tensor, pointer, bytes) of a workspace of at least ``need`` bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the call's tensors")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def _act(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError('act must be "none", "silu", "gelu" or "gelu_tanh"')
    return code


def _positions(x: torch.Tensor, name: str):
    """(B, S, C, ld) of a channels-last (B, S, C) CUDA tensor whose B * S
    positions are one stride apart."""
    sh = x.shape
    if len(sh) != 3:
        raise ValueError(f"{name} must be 3-D (samples, positions, channels)")
    B, S, C = sh
    sb, ss, sc = x.stride()
    if C > 1 and sc != 1:
        raise ValueError(f"{name} must have unit channel stride")
    ld = ss if S > 1 else sb if B > 1 else max(C, ss)
    if B > 1 and S > 0 and sb != S * ld:
        raise ValueError(f"{name}'s samples must follow one another at the stride of its positions")
    return B, S, C, ld


def _like_positions(x: torch.Tensor, ld: int, t: Optional[torch.Tensor], name: str) -> torch.Tensor:
    if t is None:
        if x.is_contiguous():
            return torch.empty_like(x)
        return torch.empty_strided(x.shape, (x.shape[1] * ld, ld, 1), dtype=x.dtype, device=x.device)
    if t.dtype is not x.dtype or t.get_device() != x.get_device() or t.shape != x.shape:
        raise ValueError(f"{name} must match x in shape, dtype and device")
    if t.stride() != x.stride() and _positions(t, name)[3] != ld and x.shape[0] * x.shape[1] > 1:
        raise ValueError(f"x and {name} must share the stride of their positions")
    return t


def _floats(t: Optional[torch.Tensor], n: int, dev: int, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(n, dtype=torch.float32, device=dev)
    if t.dtype is not torch.float32 or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {n} entries")
    return t


def _group_stats(stats: torch.Tensor, B: int, groups: int, dev: int) -> int:
    if (stats.dtype is not torch.float32 or stats.numel() != 2 * B * groups or not stats.is_contiguous()
            or stats.get_device() != dev):
        raise ValueError("stats must be a contiguous float32 CUDA tensor of shape (B, groups, 2)")
    return stats.data_ptr()


def rowops_groupnorm_act_workspace_bytes(B: int, S: int, C: int, groups: int, dtype: torch.dtype) -> int:
    return int(library().rowops_groupnorm_act_workspace_bytes(B, S, C, groups, _DTYPE_CODES.get(dtype, -1)))


def rowops_groupnorm_act(
    x: torch.Tensor,
    groups: int,
    w: Optional[torch.Tensor] = None,
    b: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    act: str = "silu",
    y: Optional[torch.Tensor] = None,
    stats: Optional[torch.Tensor] = None,
    *,
    workspace: Optional[torch.Tensor] = None,
    stream=None,
) -> torch.Tensor:
    """Group norm -> affine -> activation of channels-last ``x`` (B, S, C):
    samples, positions, channels (a channels-last image tensor of shape (B, C,
    H, W) is ``t.permute(0, 2, 3, 1).flatten(1, 2)``). ``act``: "none", "silu",
    "gelu" (exact) or "gelu_tanh". ``stats``: a float32 (B, groups, 2) tensor that
    takes (mean, rstd) for the backward pass. ``workspace``: a CUDA tensor of at
    least ``rowops_groupnorm_act_workspace_bytes(...)`` bytes, allocated per call
    when omitted."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_groupnorm_act, stream, dev, x, groups, w, b, eps, act, y, stats, workspace=workspace)
    B, S, C, ld = _positions(x, "x")
    code = _dtype_code(x)
    y = _like_positions(x, ld, y, "y")
    L = _calls or _hot_calls()
    ws, wp, wn = _scratch(workspace, L.groupnorm_act_workspace_bytes(B, S, C, groups, code), dev)
    st = L.groupnorm_act(
        x.data_ptr(), y.data_ptr(), _affine(w, x, C, dev, "w"), _affine(b, x, C, dev, "b"), eps, B, S, C, groups, ld,
        _act(act), None if stats is None else _group_stats(stats, B, groups, dev), code, wp, wn,
        _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_groupnorm_act", st)
    return y


def rowops_groupnorm_act_backward_workspace_bytes(B: int, S: int, C: int, groups: int, dtype: torch.dtype) -> int:
    return int(library().rowops_groupnorm_act_backward_workspace_bytes(B, S, C, groups, _DTYPE_CODES.get(dtype, -1)))


def rowops_groupnorm_act_backward(
    x: torch.Tensor,
    dy: torch.Tensor,
    stats: torch.Tensor,
    groups: int,
    w: Optional[torch.Tensor] = None,
    b: Optional[torch.Tensor] = None,
    act: str = "silu",
    dx: Optional[torch.Tensor] = None,
    dw: Optional[torch.Tensor] = None,
    db: Optional[torch.Tensor] = None,
    *,
    workspace: Optional[torch.Tensor] = None,
    stream=None,
):
    """Gradients of rowops_groupnorm_act for the upstream gradient ``dy`` and the
    ``stats`` that the forward call wrote: ``(dx, dw, db)``, dx as x, dw and db
    float32 (C,)."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_groupnorm_act_backward, stream, dev, x, dy, stats, groups, w, b, act, dx, dw, db,
                          workspace=workspace)
    B, S, C, ld = _positions(x, "x")
    code = _dtype_code(x)
    _like_positions(x, ld, dy, "dy")
    dx = _like_positions(x, ld, dx, "dx")
    dw = _floats(dw, C, dev, "dw")
    db = _floats(db, C, dev, "db")
    L = _calls or _hot_calls()
    ws, wp, wn = _scratch(workspace, L.groupnorm_act_backward_workspace_bytes(B, S, C, groups, code), dev)
    st = L.groupnorm_act_backward(
        x.data_ptr(), dy.data_ptr(), _affine(w, x, C, dev, "w"), _affine(b, x, C, dev, "b"),
        _group_stats(stats, B, groups, dev), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), B, S, C, groups, ld,
        _act(act), code, wp, wn, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_groupnorm_act_backward", st)
    return dx, dw, db


def _device_offset(t: Optional[torch.Tensor], dev: int):
    if t is None:
        return None
    if t.dtype is not torch.int64 or t.numel() != 1 or t.get_device() != dev:
        raise ValueError("device_offset must be an int64 CUDA tensor of one entry")
    return t.data_ptr()


def rowops_bias_dropout_residual(
    x: torch.Tensor,
    residual: Optional[torch.Tensor] = None,
    bias: Optional[torch.Tensor] = None,
    p: float = 0.1,
    seed: int = 0,
    offset: int = 0,
    y: Optional[torch.Tensor] = None,
    *,
    device_offset: Optional[torch.Tensor] = None,
    stream=None,
) -> torch.Tensor:
    """y = residual + dropout(x + bias, p) for every row of ``x`` (bias per
    column; residual laid out like x; either may be None). The mask is a function
    of (seed, offset) and the position, never stored: give each call an
    ``offset`` of its own and the backward pass the same one. ``device_offset``:
    an int64 tensor of one entry that is added to ``offset`` when the kernel
    runs, so that a captured graph replays with new masks."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_bias_dropout_residual, stream, dev, x, residual, bias, p, seed, offset, y,
                          device_offset=device_offset)
    M, N, ld, y, code, dev = _xy(x, y)
    if residual is not None and (residual.dtype is not x.dtype or residual.get_device() != dev
                                 or residual.shape != x.shape
                                 or (residual.stride() != x.stride()
                                     and (M > 1 or (M == 1 and N > 1 and residual.stride(1) != 1)))):
        raise ValueError("residual must match x in shape, dtype, device and row stride")
    st = (_calls or _hot_calls()).bias_dropout_residual(
        x.data_ptr(), None if residual is None else residual.data_ptr(), _affine(bias, x, N, dev, "bias"),
        y.data_ptr(), p, seed, offset, _device_offset(device_offset, dev), M, N, ld, code, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_bias_dropout_residual", st)
    return y


def rowops_bias_dropout_residual_backward_workspace_bytes(M: int, N: int, dtype: torch.dtype) -> int:
    return int(library().rowops_bias_dropout_residual_backward_workspace_bytes(M, N, _DTYPE_CODES.get(dtype, -1)))


def rowops_bias_dropout_residual_backward(
    dy: torch.Tensor,
    p: float = 0.1,
    seed: int = 0,
    offset: int = 0,
    dx: Optional[torch.Tensor] = None,
    dbias: Optional[torch.Tensor] = None,
    bias_grad: bool = True,
    *,
    device_offset: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
    stream=None,
):
    """Gradients of rowops_bias_dropout_residual for the upstream gradient ``dy``
    and the forward call's p, seed and offsets: ``(dx, dbias)``, dx as dy (and
    may be ``dy``), dbias float32 (N,), or None without ``bias_grad``. The
    residual's gradient is dy itself."""
    dev = dy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_bias_dropout_residual_backward, stream, dev, dy, p, seed, offset, dx, dbias,
                          bias_grad, device_offset=device_offset, workspace=workspace)
    M, N, ld, dx, code, dev = _xy(dy, dx)
    L = _calls or _hot_calls()
    ws, wp, wn = None, None, 0
    if bias_grad:
        dbias = _floats(dbias, N, dev, "dbias")
        need = L.bias_dropout_residual_backward_workspace_bytes(M, N, code)
        ws, wp, wn = _scratch(workspace, need, dev)
    elif dbias is not None:
        raise ValueError("dbias is given but bias_grad is false")
    st = L.bias_dropout_residual_backward(
        dy.data_ptr(), dx.data_ptr(), None if dbias is None else dbias.data_ptr(), p, seed, offset,
        _device_offset(device_offset, dev), M, N, ld, code, wp, wn, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_bias_dropout_residual_backward", st)
    return dx, dbias


def rowops_router_balance_loss_workspace_bytes(T: int, E: int, dtype: torch.dtype) -> int:
    return int(library().rowops_router_balance_loss_workspace_bytes(T, E, _DTYPE_CODES.get(dtype, -1)))


def _row_mask(mask: Optional[torch.Tensor], T: int, dev: int):
    if mask is None:
        return None
    if (mask.dtype not in (torch.bool, torch.uint8) or mask.numel() != T or not mask.is_contiguous()
            or mask.get_device() != dev):
        raise ValueError("mask must be a contiguous bool or uint8 CUDA tensor of one entry a row")
    return mask.data_ptr()


def _counts(counts: Optional[torch.Tensor], E: int, dev: int) -> torch.Tensor:
    if counts is None:
        return torch.empty(E + 1, dtype=torch.int64, device=dev)
    if (counts.dtype is not torch.int64 or counts.numel() != E + 1 or not counts.is_contiguous()
            or counts.get_device() != dev):
        raise ValueError("counts must be a contiguous int64 CUDA tensor of E + 1 entries")
    return counts


def rowops_router_balance_loss(
    logits: torch.Tensor,
    experts: torch.Tensor,
    coef: float = 0.01,
    mask: Optional[torch.Tensor] = None,
    loss: Optional[torch.Tensor] = None,
    counts: Optional[torch.Tensor] = None,
    *,
    workspace: Optional[torch.Tensor] = None,
    stream=None,
):
    """Balance loss of a router from its ``logits`` (T, E) and the chosen
    ``experts`` (T, K) (int32 or int64): ``(loss, counts)``, loss float32 (1,),
    counts int64 (E + 1,): the experts' counts and, last, the rows that took
    part. ``mask``: bool or uint8 (T,), rows with 0 take no part. The counts enter
    divided by the choices, T K of them, so that an even load gives ``coef`` (a
    coefficient made for a definition without that K is to be multiplied by it)."""
    dev = logits.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_router_balance_loss, stream, dev, logits, experts, coef, mask, loss, counts,
                          workspace=workspace)
    T, E, ld = _rows(logits, "logits")
    code = _dtype_code(logits)
    if experts.dim() != 2 or experts.shape[0] != T or not experts.is_contiguous() or experts.get_device() != dev:
        raise ValueError("experts must be a contiguous (T, K) tensor on the device of the logits")
    width = {torch.int64: 8, torch.int32: 4}.get(experts.dtype)
    if width is None:
        raise TypeError(f"experts must be int32 or int64, not {experts.dtype}")
    loss = _floats(loss, 1, dev, "loss")
    counts = _counts(counts, E, dev)
    L = _calls or _hot_calls()
    ws, wp, wn = _scratch(workspace, L.router_balance_loss_workspace_bytes(T, E, code), dev)
    st = L.router_balance_loss(
        logits.data_ptr(), experts.data_ptr(), width, _row_mask(mask, T, dev), coef, loss.data_ptr(),
        counts.data_ptr(), T, E, experts.shape[1], ld, code, wp, wn, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_router_balance_loss", st)
    return loss, counts


def rowops_router_balance_loss_backward(
    logits: torch.Tensor,
    counts: torch.Tensor,
    top_k: int,
    dloss: torch.Tensor,
    coef: float = 0.01,
    mask: Optional[torch.Tensor] = None,
    dlogits: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """Gradient of rowops_router_balance_loss with respect to the logits, for the
    forward call's ``counts``, coef and mask, the choices per row ``top_k`` and
    the loss's own gradient ``dloss`` (float32, one entry, on the GPU).
    ``dlogits`` may be ``logits``."""
    dev = logits.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_router_balance_loss_backward, stream, dev, logits, counts, top_k, dloss, coef, mask,
                          dlogits)
    T, E, ld, dlogits, code, dev = _xy(logits, dlogits)
    if dloss.dtype is not torch.float32 or dloss.numel() != 1 or dloss.get_device() != dev:
        raise ValueError("dloss must be a float32 CUDA tensor of one entry")
    st = (_calls or _hot_calls()).router_balance_loss_backward(
        logits.data_ptr(), _counts(counts, E, dev).data_ptr(), dloss.data_ptr(), _row_mask(mask, T, dev), coef,
        dlogits.data_ptr(), T, E, top_k, ld, code, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_router_balance_loss_backward", st)
    return dlogits


# ---------------------------------------------------------------------------
# Serving operators: RMSNorm with an 8-bit result, attention of one new token
# over a paged cache, sampling. Devices and streams as for the training operators.
# ---------------------------------------------------------------------------
_E4M3 = torch.float8_e4m3fn


def rowops_rmsnorm_quant(
    x: torch.Tensor,
    residual: Optional[torch.Tensor] = None,
    w: Optional[torch.Tensor] = None,
    eps: float = 1e-5,
    group: int = 0,
    q: Optional[torch.Tensor] = None,
    scales: Optional[torch.Tensor] = None,
    residual_out: Optional[torch.Tensor] = None,
    *,
    stream=None,
):
    """RMSNorm of ``x`` (+ ``residual``) in 8 bits: ``(q, scales, residual_out)`` with
    q float8_e4m3fn (M, N), scales float32 (M, groups), one for every ``group``
    columns (a multiple of 32; 0: one a row), so that the norm is about q * scale,
    and residual_out = x + residual (None without a residual), which may be ``x``
    or ``residual`` themselves. A given ``q`` may have a row stride of its own. The
    products of rows and ``w`` have to stay in fp32's range."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_rmsnorm_quant, stream, dev, x, residual, w, eps, group, q, scales, residual_out)
    sh, xs, dt = x.shape, x.stride(), x.dtype
    if len(sh) != 2:
        raise ValueError("x must be 2-D (M, N)")
    M, N = sh
    if N > 0 and xs[1] != 1:
        raise ValueError("x must have unit column stride")
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"rowops supports float32 and bfloat16, not {dt}")
    whole = x.is_contiguous()
    pr = po = None
    if residual is not None:
        if residual.dtype is not dt or residual.get_device() != dev or residual.shape != sh:
            raise ValueError("residual must match x in shape, dtype and device")
        if residual.stride() != xs and (M > 1 or (M == 1 and N > 1 and residual.stride(1) != 1)):
            raise ValueError("x and residual must share the row stride")
        if residual_out is None and whole:
            residual_out = torch.empty_like(x)
        else:
            residual_out = _out_like(x, residual_out)
        pr, po = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out is given but residual is not")
    groups = 1 if group <= 0 else -(-N // group)
    if q is None:
        q = torch.empty_like(x, dtype=_E4M3) if whole else torch.empty(M, N, dtype=_E4M3, device=x.device)
        ldq = N
    else:
        if q.dtype is not _E4M3 or q.shape != sh or q.get_device() != dev or (N > 1 and q.stride(1) != 1):
            raise ValueError("q must be a float8_e4m3fn CUDA tensor of x's shape with unit column stride")
        ldq = q.stride(0) if M > 1 else max(N, q.stride(0))
    if scales is None:
        scales = torch.empty((M, groups), dtype=torch.float32, device=x.device)
    else:
        _floats(scales, M * groups, dev, "scales")
    st = (_calls or _hot_calls()).rmsnorm_quant(
        x.data_ptr(), pr, q.data_ptr(), scales.data_ptr(), po, _affine(w, x, N, dev, "w"), eps, M, N,
        xs[0] if M > 1 else max(N, xs[0]), ldq, group, code, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_rmsnorm_quant", st)
    return q, scales, residual_out


def _heads(t: torch.Tensor, name: str):
    """(B, heads, D, stride of a sequence) of a (B, heads, D) tensor, head after head."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D (sequences, heads, D)")
    B, H, D = t.shape
    sb, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}'s heads must follow one another")
    return B, H, D, (sb if B > 1 else max(H * D, sb))


def rowops_paged_attention_workspace_bytes(B: int, heads: int, kv_heads: int, D: int, page: int, max_pages: int,
                                           window: int, dtype: torch.dtype) -> int:
    return int(library().rowops_paged_attention_workspace_bytes(B, heads, kv_heads, D, page, max_pages, window,
                                                                _DTYPE_CODES.get(dtype, -1)))


def rowops_paged_attention(
    q: torch.Tensor,
    k_cache: torch.Tensor,
    v_cache: torch.Tensor,
    page_table: torch.Tensor,
    lengths: torch.Tensor,
    scale: Optional[float] = None,
    window: int = 0,
    out: Optional[torch.Tensor] = None,
    lse: Optional[torch.Tensor] = None,
    *,
    workspace: Optional[torch.Tensor] = None,
    stream=None,
) -> torch.Tensor:
    """Attention of one new token a sequence, ``q`` (B, heads, D), over paged caches
    ``k_cache``, ``v_cache`` (pages, slots, kv_heads, D) (any strides, the same in both,
    with unit stride in D). ``page_table`` int32 (B, max_pages) names the pages of a
    sequence's positions in turn, ``lengths`` int32 (B,) its positions, the new token's
    among them. ``scale``: 1 / sqrt(D) when None; ``window``: only that many last
    positions (0: all); ``lse``: a float32 (B, heads) tensor that takes the logarithm of
    the sum of exponentials. ``workspace``: a CUDA tensor of at least
    ``rowops_paged_attention_workspace_bytes(...)`` bytes, allocated per call when
    omitted."""
    dev = q.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_paged_attention, stream, dev, q, k_cache, v_cache, page_table, lengths, scale, window,
                          out, lse, workspace=workspace)
    B, H, D, ldq = _heads(q, "q")
    code = _dtype_code(q)
    ks, dt = k_cache.shape, q.dtype
    if len(ks) != 4 or ks != v_cache.shape or ks[3] != D:
        raise ValueError("k_cache and v_cache must both be (pages, slots, kv_heads, D)")
    if (k_cache.dtype is not dt or v_cache.dtype is not dt or k_cache.get_device() != dev
            or v_cache.get_device() != dev):
        raise ValueError("k_cache and v_cache must match q in dtype and device")
    kt, vt = k_cache.stride(), v_cache.stride()
    if kt != vt and any(n > 1 and a != b for n, a, b in zip(ks, kt, vt)):
        raise ValueError("k_cache and v_cache must share their strides")
    if D > 1 and kt[3] != 1:
        raise ValueError("k_cache and v_cache must have unit stride in D")
    ts = page_table.shape
    if len(ts) != 2 or ts[0] != B or (ts[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be (B, max_pages) with unit column stride")
    if lengths.shape != (B,) or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous (B,) tensor")
    if (page_table.dtype is not torch.int32 or lengths.dtype is not torch.int32 or page_table.get_device() != dev
            or lengths.get_device() != dev):
        raise ValueError("page_table and lengths must be int32 CUDA tensors on the device of the call's tensors")
    width = ts[1]
    if out is None:
        out = torch.empty_like(q) if ldq == H * D and q.is_contiguous() else torch.empty(B, H, D, dtype=dt, device=q.device)
        ldo = H * D
    else:
        if out.dtype is not dt or out.shape != q.shape or out.get_device() != dev:
            raise ValueError("out must match q in shape, dtype and device")
        ldo = _heads(out, "out")[3]
    L = _calls or _hot_calls()
    ws, wp, wn = _scratch(workspace, L.paged_attention_workspace_bytes(B, H, ks[2], D, ks[1], width, window, code), dev)
    st = L.paged_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), out.data_ptr(),
        None if lse is None else _floats(lse, B * H, dev, "lse").data_ptr(), max(D, 1) ** -0.5 if scale is None else scale,
        window, B, H, ks[2], D, ldq, ldo, ks[0], ks[1], kt[0], kt[1], kt[2], width,
        page_table.stride(0) if B > 1 else max(width, page_table.stride(0)), code, wp, wn, _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_paged_attention", st)
    return out


def _knob(v, M: int, dtype: torch.dtype, dev: int, name: str):
    """(device pointer, number) of a number for every row or one a row."""
    if isinstance(v, torch.Tensor):
        if v.dtype is not dtype or v.shape != (M,) or not v.is_contiguous() or v.get_device() != dev:
            raise ValueError(f"{name} must be a number or a contiguous {dtype} CUDA tensor of one entry a row")
        return v.data_ptr(), 0
    return None, v


def rowops_sample(
    logits: torch.Tensor,
    u: torch.Tensor,
    temperature=1.0,
    top_k=0,
    top_p=1.0,
    min_p=0.0,
    token: Optional[torch.Tensor] = None,
    logprob: Optional[torch.Tensor] = None,
    *,
    stream=None,
) -> torch.Tensor:
    """One token a row of ``logits`` (M, N), drawn with the uniform numbers ``u``
    (float32 (M,), in [0, 1)): int64 (M,). ``temperature`` (0: the maximum), ``top_k``
    (0: off), ``top_p`` (1: off; of what top-k keeps) and ``min_p`` (0: off; of the
    maximum's weight) are numbers, or tensors of one entry a row (float32; top_k int32).
    ``logprob``: a float32 (M,) tensor that takes the tokens' log-probabilities among
    what is kept. A row with a NaN, or of -inf alone, gives -1."""
    dev = logits.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(rowops_sample, stream, dev, logits, u, temperature, top_k, top_p, min_p, token, logprob)
    M, N, ld = _rows(logits, "logits")
    f32 = torch.float32
    if u.dtype is not f32 or u.shape != (M,) or not u.is_contiguous() or u.get_device() != dev:
        raise ValueError("u must be a contiguous float32 CUDA tensor of one entry a row")
    if token is None:
        token = torch.empty(M, dtype=torch.int64, device=logits.device)
    elif token.dtype is not torch.int64 or token.shape != (M,) or not token.is_contiguous() or token.get_device() != dev:
        raise ValueError("token must be a contiguous int64 CUDA tensor of one entry a row")
    if not isinstance(top_k, torch.Tensor):
        top_k = min(max(top_k, -1), N)  # (32 bits in the call)
    st = (_calls or _hot_calls()).sample(
        logits.data_ptr(), u.data_ptr(), *_knob(temperature, M, f32, dev, "temperature"),
        *_knob(top_k, M, torch.int32, dev, "top_k"), *_knob(top_p, M, f32, dev, "top_p"),
        *_knob(min_p, M, f32, dev, "min_p"), token.data_ptr(),
        None if logprob is None else _floats(logprob, M, dev, "logprob").data_ptr(), M, N, ld, _dtype_code(logits),
        _current_raw_stream(dev))
    if st:
        raise RowopsError("rowops_sample", st)
    return token
