"""MXFP4 rows and the experts' products on them (OCP Microscaling Formats 1.0).

    codes, scales = quantize_fp4(x)                                    # bf16 [..][K] to 4 bits
    h, hs = expert_swiglu_fp4(codes, scales, w13, w13_scales, counts=..., offsets=...)   # FP4 rows again
    y = expert_gemm_fp4(h, hs, w2, w2_scales, counts=..., offsets=...)                   # bf16, what combine reads

Codes are uint8 [..][K / 2], two e2m1 codes a byte with the lower channel in the lower half; scales are uint8 [..][K / 32],
E8M0: 2^(byte - 127), 255 a NaN.  Weights are codes [E][N][K / 2] and scales [E][N][K / 32].  The rows come in the layouts
of expert_gemm; K is a multiple of 128.  Context.quantize_fp4, dispatch_permuted_fp4, expert_swiglu_fp4 and
expert_gemm_fp4 run them over a dispatch.
"""
from __future__ import annotations

import torch

from .experts import _GROUPS, _ROWS, _WEIGHT, _call, _empty, _output, _refuse, _status_ptr, _step, _stream_of

_U8, _I32, _BF16 = torch.uint8, torch.int32, torch.bfloat16


def fp4_row_views(rows: torch.Tensor, channels: int):
    """(codes, scales) of FP4 rows [rows][row bytes]: channels / 2 bytes of codes, then channels / 32 scales."""
    return rows[:, :channels // 2], rows[:, channels // 2:channels // 2 + channels // 32]


def quantize_fp4(x, out=None, stream=None):
    """(codes [..][K/2], scales [..][K/32]) of bf16 rows [rows][K] or [E][rows][K], K a multiple of 128."""
    index, shape = x.get_device(), x.shape
    if index < 0:
        _refuse("quantize_fp4: all tensors must be on a CUDA device")
    if x.dtype != _BF16 or len(shape) not in (2, 3) or shape[-1] == 0 or shape[-1] % 128:
        _refuse(f"quantize_fp4: bf16 rows [rows][K] or [E][rows][K], K a multiple of 128: got {x.dtype} {tuple(shape)}")
    k = shape[-1]
    if out is None:
        cs, ss = k // 2, k // 32
        codes, scales = _empty(x, stream, (*shape[:-1], cs), _U8), _empty(x, stream, (*shape[:-1], ss), _U8)
    else:
        codes, scales = out
        cs = _output("quantize_fp4: out codes", codes, shape, k // 2, (_U8,), index)
        ss = _output("quantize_fp4: out scales", scales, shape, k // 32, (_U8,), index)
    _call("ep_quantize_fp4", index, x.data_ptr(), _step("quantize_fp4: x", x), x.numel() // k, k, codes.data_ptr(), cs, scales.data_ptr(), ss,
          _stream_of(stream, index))
    return codes, scales


def _products(name, x, x_scales, w, w_scales, counts, offsets, bases, expected):
    """(device index, row shape, weight rows, the three C descriptors) of one product, all checked."""
    index = x.get_device()
    xs, ws = x.shape, w.shape
    lead, dims = len(xs), len(ws)
    if index < 0:
        _refuse(f"{name}: all tensors must be on a CUDA device")
    if lead not in (2, 3) or x.dtype != _U8 or xs[-1] == 0 or xs[-1] % 64:
        _refuse(f"{name}: codes uint8 [rows][K/2] or [E][rows][K/2], K a multiple of 128: got {x.dtype} {tuple(xs)}")
    half = xs[-1]
    per = half // 16
    ss = x_scales.shape
    if x_scales.dtype != _U8 or len(ss) != lead or ss[-1] != per or ss[0] != xs[0] or ss[-2] != xs[-2]:
        _refuse(f"{name}: scales uint8 {(*xs[:-1], per)}: got {x_scales.dtype} {tuple(ss)}")
    if dims not in (2, 3) or w.dtype != _U8 or ws[-1] != half or not w.is_contiguous():
        _refuse(f"{name}: weight codes uint8 [E][N][{half}] or [N][{half}], contiguous: got {w.dtype} {tuple(ws)}")
    n, groups = ws[-2], ws[0] if dims == 3 else 1
    ss = w_scales.shape
    if w_scales.dtype != _U8 or ss != (*ws[:-1], per) or not w_scales.is_contiguous():
        _refuse(f"{name}: weight scales uint8 {(*ws[:-1], per)}, contiguous: got {w_scales.dtype} {tuple(ss)}")
    if x_scales.get_device() != index or w.get_device() != index or w_scales.get_device() != index:
        _refuse(f"{name}: all tensors must be on the same CUDA device")
    counts_at = offsets_at = bases_at = per_base = 0
    if counts is not None:
        if counts.dtype != _I32 or counts.numel() != groups or not counts.is_contiguous() or counts.get_device() != index:
            _refuse(f"{name}: counts int32 [{groups}], contiguous, on the same device")
        counts_at = counts.data_ptr()
    if offsets is not None:
        if offsets.dtype != _I32 or offsets.numel() != groups or not offsets.is_contiguous() or offsets.get_device() != index:
            _refuse(f"{name}: offsets int32 [{groups}], contiguous, on the same device")
        offsets_at = offsets.data_ptr()
    rows = stride = xs[0]
    if lead == 3:
        if rows != groups or offsets is not None:
            _refuse(f"{name}: {rows} regions for {groups} weights, which take no offsets")
        stride = xs[1]
        rows *= stride
    elif groups != 1 and (counts is None or offsets is None):
        _refuse(f"{name}: {groups} groups need counts and offsets")
    if bases is not None:
        runs = bases.numel() - 1
        if bases.dtype != _I32 or runs < 1 or groups % runs or not bases.is_contiguous() or bases.get_device() != index:
            _refuse(f"{name}: bases int32 [R + 1] for {groups} groups in R equal runs, contiguous, on the same device")
        bases_at, per_base = bases.data_ptr(), groups // runs
    return (index, xs, n, _ROWS(x.data_ptr(), _step(name, x), x_scales.data_ptr(), _step(name, x_scales), rows),
            _GROUPS(counts_at, offsets_at, bases_at, per_base, stride, expected), _WEIGHT(w.data_ptr(), w_scales.data_ptr(), groups, n, 2 * half))


def expert_gemm_fp4(x, x_scales, w, w_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None, expected_rows=0):
    """y = x w^T per expert: bf16 [rows][N] (or [E][cap][N]).  Rows of no expert are not written.  Arguments as expert_gemm's."""
    index, shape, n, cx, cg, cw = _products("expert_gemm_fp4", x, x_scales, w, w_scales, counts, offsets, bases, expected_rows)
    step = n
    if out is None:
        out = _empty(x, stream, (*shape[:-1], n), _BF16)
    else:
        step = _output("expert_gemm_fp4: out", out, shape, n, (_BF16,), index)
    _call("ep_expert_gemm_fp4", index, cx, cg, cw, out.data_ptr(), step, _status_ptr(status, index), _stream_of(stream, index))
    return out


def expert_swiglu_fp4(x, x_scales, w13, w13_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None,
                      expected_rows=0):
    """silu(x wg^T) * (x wu^T) per expert, w13 = [gate; up] [E][2I][K/2], requantised: (codes [rows][I/2], scales [rows][I/32])
    (or [E][cap][..])."""
    index, shape, n, cx, cg, cw = _products("expert_swiglu_fp4", x, x_scales, w13, w13_scales, counts, offsets, bases, expected_rows)
    if n % 256:
        _refuse(f"expert_swiglu_fp4: {n} weight rows are no gate and up of a multiple of 128 each")
    inter = n // 2
    if out is None:
        cs, ss = inter // 2, inter // 32
        codes, scales = _empty(x, stream, (*shape[:-1], cs), _U8), _empty(x, stream, (*shape[:-1], ss), _U8)
    else:
        codes, scales = out
        cs = _output("expert_swiglu_fp4: out codes", codes, shape, inter // 2, (_U8,), index)
        ss = _output("expert_swiglu_fp4: out scales", scales, shape, inter // 32, (_U8,), index)
    _call("ep_expert_swiglu_fp4", index, cx, cg, cw, codes.data_ptr(), cs, scales.data_ptr(), ss, _status_ptr(status, index),
          _stream_of(stream, index))
    return codes, scales
