"""The norm before a layer: residual addition, RMS norm, and what the router and dispatch read of it.

    got = rms_norm(x, weight, residual=r, fp8=True)      # got["y"] bf16, got["residual"] = x + r, got["rows"] FP8 rows
    dx, dweight = rms_norm_backward(dy, got["residual"], weight, dresidual=dr)

x, y and dy are bf16 rows [..][H] (up to three dimensions, rows evenly spaced); the residual is bf16 or fp32, and so is
the weight.  The FP8 rows are those of Context.quantize_fp8: what dispatch_fp8 and dispatch_permuted_fp8 carry.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from .experts import _call, _empty, _entry, _refuse, _step, _stream_of

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_TYPES = {_BF16: 0, _F32: 1}


def _rows(name, t, shape, dtypes, index):
    """Elements between the rows of a row array of this shape."""
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != index:
        _refuse(f"{name}: {' or '.join(str(d) for d in dtypes)} {tuple(shape)} on the same CUDA device: got {t.dtype} {tuple(t.shape)}")
    if len(shape) == 1:
        if not t.is_contiguous():
            _refuse(f"{name}: channels must be contiguous (strides {t.stride()})")
        return shape[0]
    return _step(name, t)


def _made(name, given, like, stream, shape, dtype, index):
    """(output, elements between its rows): the given one, checked, or a new one on `like`'s device."""
    if given is None:
        return _empty(like, stream, shape, dtype), shape[-1]
    return given, _rows(name, given, shape, (dtype,), index)


def _inputs(name, x, weight):
    """(device index, shape, rows, channels) of a norm's rows and its weight, both checked."""
    index, shape = x.get_device(), x.shape
    if index < 0:
        _refuse(f"{name}: all tensors must be on a CUDA device")
    if not 1 <= len(shape) <= 3 or shape[-1] == 0:
        _refuse(f"{name}: rows [..][H] of up to three dimensions: got {tuple(shape)}")
    hidden = shape[-1]
    if weight.dtype not in _TYPES or weight.shape != (hidden,) or not weight.is_contiguous() or weight.get_device() != index:
        _refuse(f"{name}: weight bf16 or fp32 [{hidden}], contiguous, on the same device: got {weight.dtype} {tuple(weight.shape)}")
    return index, shape, x.numel() // hidden, hidden


def rms_norm(x, weight, eps=1e-6, residual=None, y=True, fp8=False, out=None, stream=None) -> dict:
    """RMS norm of h = x + residual: {"y": bf16 [..][H], "residual": h (with a residual), "rows": FP8 rows [rows][row bytes]}.

    y, fp8: which outputs to make.  out: a dict with some of them to write into; "residual" may be the residual itself and
    "y" may be x, so that nothing is allocated."""
    index, shape, rows, hidden = _inputs("rms_norm", x, weight)
    given = {} if out is None else out
    got = {}
    sx = _rows("rms_norm: x", x, shape, (_BF16,), index)
    rt = sr = so = sy = sq = 0
    r_at = o_at = y_at = q_at = None  # without an output: no array
    if residual is not None:
        kind = residual.dtype
        sr = _rows("rms_norm: residual", residual, shape, (_BF16, _F32), index)
        rt, r_at = _TYPES[kind], residual.data_ptr()
        got["residual"], so = _made("rms_norm: out residual", given.get("residual"), x, stream, shape, kind, index)
        o_at = got["residual"].data_ptr()
    elif given.get("residual") is not None:
        _refuse("rms_norm: an output for the residual, but no residual")
    if y or given.get("y") is not None:
        got["y"], sy = _made("rms_norm: out y", given.get("y"), x, stream, shape, _BF16, index)
        y_at = got["y"].data_ptr()
    if fp8 or given.get("rows") is not None:
        if hidden % 128:
            _refuse(f"rms_norm: FP8 rows of {hidden} channels (a multiple of 128)")
        size = (hidden + hidden // 32 + 15) // 16 * 16
        got["rows"], sq = _made("rms_norm: out rows", given.get("rows"), x, stream, (rows, size), _U8, index)
        q_at = got["rows"].data_ptr()
    _call("ep_rms_norm", index, x.data_ptr(), sx, r_at, sr, rt, weight.data_ptr(), _TYPES[weight.dtype], eps, rows, hidden, o_at, so, y_at, sy,
          q_at, sq, _stream_of(stream, index))
    return got


def rms_norm_backward(dy, h, weight, eps=1e-6, dresidual=None, out=None, workspace=None, stream=None):
    """(dx, dweight) of rms_norm: dy bf16, the gradient of its output; h: what it took the norm of (its "residual" output,
    or x without one); dresidual, of h's type: the gradient that reaches h from elsewhere.

    dx, of h's type, is the gradient of x and of the residual alike; dweight is fp32.  out: (dx, dweight) to write into,
    dx may be dresidual.  `workspace` (contiguous, rms_norm_backward_workspace bytes) is allocated when it is not given."""
    index, shape, rows, hidden = _inputs("rms_norm_backward", h, weight)
    sh = _rows("rms_norm_backward: h", h, shape, (_BF16, _F32), index)
    sg = _rows("rms_norm_backward: dy", dy, shape, (_BF16,), index)
    sd = 0 if dresidual is None else _rows("rms_norm_backward: dresidual", dresidual, shape, (h.dtype,), index)
    dx, dweight = (None, _empty(h, stream, (hidden,), _F32)) if out is None else out
    dx, so = _made("rms_norm_backward: out dx", dx, h, stream, shape, h.dtype, index)
    if dweight.dtype != _F32 or dweight.shape != (hidden,) or not dweight.is_contiguous() or dweight.get_device() != index:
        _refuse(f"rms_norm_backward: out dweight fp32 [{hidden}], contiguous, on the same device")
    if workspace is None:
        workspace = _empty(h, stream, (_workspace_bytes("ep_rms_norm_backward_workspace", index, rows, hidden),), _U8)
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        _refuse("rms_norm_backward: workspace must be contiguous, on the same device")
    _call("ep_rms_norm_backward", index, dy.data_ptr(), sg, h.data_ptr(), sh, _TYPES[h.dtype], weight.data_ptr(), _TYPES[weight.dtype], eps,
          None if dresidual is None else dresidual.data_ptr(), sd, rows, hidden, dx.data_ptr(), so, dweight.data_ptr(), workspace.data_ptr(),
          workspace.nbytes, _stream_of(stream, index))
    return dx, dweight


def rms_norm_backward_workspace(rows: int, hidden: int) -> int:
    """Bytes of workspace rms_norm_backward needs on the current device (0 for sizes it refuses)."""
    return int(_lib.load().ep_rms_norm_backward_workspace(rows, hidden))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, index: int, *args) -> int:
    with torch.cuda.device(index):
        return int(_entry(name)(*args))
