"""The experts' side of the path: what runs between dispatch and combine.

    h, hs = expert_swiglu(x, xs, w13, w13_scales, counts=..., offsets=...)   # silu(x wg^T) * (x wu^T), FP8 rows
    y = expert_gemm(h, hs, w2, w2_scales, counts=..., offsets=...)           # bf16 rows, what combine reads

x and h are e4m3 codes (uint8 or float8_e4m3fn) with one fp32 scale per 128
channels; weights are codes [E][N][K] with one scale per 128 x 128 block.  The
rows come as one of

* [rows][K] with counts [E] and offsets [E] (int32, on the GPU): expert e has the
  rows offsets[e] .. offsets[e] + counts[e] - 1 (the permuted layout),
* [E][cap][K] with counts [E]: the first counts[e] rows of each region (the
  packed low-latency layout), or all of them without counts,
* [rows][K] with a 2-D weight: one dense product.

    out = moe_tokens(x, topk_idx, topk_weights, w13, w2, w13_scales, w2_scales)   # a whole layer, up to 64 tokens

Context.expert_swiglu / expert_gemm and LLBuffer.expert_swiglu / expert_gemm
take the groups from the dispatch handle and the packed dict.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _lib
from ._lib import EpError, check

_U8, _E4M3, _F32, _I32, _BF16 = torch.uint8, torch.float8_e4m3fn, torch.float32, torch.int32, torch.bfloat16
_CODES = (_U8, _E4M3)
# bits of a status word, as the C entry points OR them in, by the status a check raises first
_STATUS_BITS = ((1, -2, "topk_idx holds a value outside [-1, E)"), (4, -4, "a bounded device wait ran out"),
                (2, -3, "a group's rows lie outside the row arrays"))

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status word for the calls of this module."""
    return torch.zeros(1, dtype=torch.int32, device=device if device is not None else "cuda")


def check_status(status: torch.Tensor) -> None:
    """Reads (waits for) and clears a status word; raises EpError for the bits set."""
    bits = int(status.item())
    if bits:
        status.zero_()
        for bit, code, text in _STATUS_BITS:
            if bits & bit:
                raise EpError("check_status", code, text)
        raise EpError("check_status", -5, f"device status bits {bits:#x}")


def fp8_row_views(rows: torch.Tensor, channels: int):
    """(codes, scales) of FP8 rows [rows][row bytes]: `channels` e4m3 codes, then channels / 128 fp32 scales."""
    return rows[:, :channels], rows[:, channels:channels + channels // 32].view(torch.float32)


# The calls below are a few microseconds of kernel at their smallest, so their checks read each property
# once and build a message only when they refuse.

def _stream_of(stream, index: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _refuse(text: str):
    raise ValueError(text)


def _step(name: str, t: torch.Tensor) -> int:
    """Elements between the rows of t [rows][n] or [E][rows][n], whose rows have to be evenly spaced."""
    n = t.shape[-1]
    if t.is_contiguous():
        return n
    shape, st = t.shape, t.stride()
    if n > 1 and st[-1] != 1:
        _refuse(f"{name}: channels must be contiguous (strides {st})")
    if len(shape) == 2:
        return st[0] if shape[0] > 1 else max(st[0], n)
    if shape[1] > 1:
        if shape[0] > 1 and st[0] != shape[1] * st[1]:
            _refuse(f"{name}: regions must be evenly spaced (strides {st})")
        return st[1]
    return st[0] if shape[0] > 1 else max(st[0], n)


# ep_fp8_rows, ep_row_groups, ep_fp8_weight and ep_moe_weights as the C side lays them out
_ROWS, _GROUPS, _WEIGHT = struct.Struct("@PqPqq").pack, struct.Struct("@PPPiqq").pack, struct.Struct("@PPiii0P").pack
_MOE = struct.Struct("@PPPPiii0P").pack


def _products(name, x, x_scales, w, w_scales, counts, offsets, bases, expected):
    """(device index, row shape, weight rows, the three C descriptors) of one product, all checked."""
    index = x.get_device()
    xs, ws = x.shape, w.shape
    lead, dims = len(xs), len(ws)
    if index < 0:
        _refuse(f"{name}: all tensors must be on a CUDA device")
    if lead not in (2, 3) or x.dtype not in _CODES or xs[-1] == 0 or xs[-1] % 128:
        _refuse(f"{name}: codes [rows][K] or [E][rows][K], uint8 or e4m3, K a multiple of 128: got {x.dtype} {tuple(xs)}")
    k = xs[-1]
    kb = k // 128
    ss = x_scales.shape
    if x_scales.dtype != _F32 or len(ss) != lead or ss[-1] != kb or ss[0] != xs[0] or ss[-2] != xs[-2]:
        _refuse(f"{name}: fp32 scales {(*xs[:-1], kb)}: got {x_scales.dtype} {tuple(ss)}")
    if dims not in (2, 3) or w.dtype not in _CODES or ws[-1] != k or not w.is_contiguous():
        _refuse(f"{name}: weight codes [E][N][{k}] or [N][{k}], uint8 or e4m3, contiguous: got {w.dtype} {tuple(ws)}")
    n, groups = ws[-2], ws[0] if dims == 3 else 1
    ss = w_scales.shape
    if (w_scales.dtype != _F32 or len(ss) != dims or ss[-1] != kb or ss[-2] != (n + 127) // 128 or (dims == 3 and ss[0] != groups)
            or not w_scales.is_contiguous()):
        _refuse(f"{name}: weight scales fp32 {(*ws[:-2], (n + 127) // 128, kb)}, contiguous: got {w_scales.dtype} {tuple(ss)}")
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
            _GROUPS(counts_at, offsets_at, bases_at, per_base, stride, expected), _WEIGHT(w.data_ptr(), w_scales.data_ptr(), groups, n, k))


def _status_ptr(status, index: int):
    if status is None or isinstance(status, int):  # an address: the status word of a context or a buffer
        return status
    if status.dtype != _I32 or status.numel() < 1 or status.get_device() != index:
        _refuse("status: an int32 word on the same device")
    return status.data_ptr()


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    return getattr(_lib.load(), name)


def _call(name: str, index: int, *args):
    """The C entry point with the tensors' device current."""
    if _current_device() == index:
        code = _entry(name)(*args)
    else:
        with torch.cuda.device(index):
            code = _entry(name)(*args)
    if code:
        check(name, code)


def _empty(like, stream, shape, dtype):
    """A tensor on `like`'s device, allocated for `stream`."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _output(name, t, like, n, dtypes, index):
    """Elements between the rows of an output with `like`'s rows and n channels."""
    shape = t.shape
    if (len(shape) != len(like) or shape[-1] != n or shape[0] != like[0] or shape[-2] != like[-2] or t.dtype not in dtypes
            or t.get_device() != index):
        _refuse(f"{name}: {dtypes[0]} {(*like[:-1], n)} on the same device: got {t.dtype} {tuple(shape)}")
    return _step(name, t)


def expert_gemm(x, x_scales, w, w_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None, expected_rows=0):
    """y = x w^T per expert: bf16 [rows][N] (or [E][cap][N]).  Rows of no expert are not written.

    bases: int32 [R + 1], added to the offsets of R equal runs of experts (a dispatch handle's perm_rank_base).
    expected_rows: about how many rows an expert has, where the caller knows; it only chooses the kernel's shape."""
    index, shape, n, cx, cg, cw = _products("expert_gemm", x, x_scales, w, w_scales, counts, offsets, bases, expected_rows)
    if out is None:
        out = _empty(x, stream, (*shape[:-1], n), _BF16)
    _call("ep_expert_gemm", index, cx, cg, cw, out.data_ptr(), _output("expert_gemm: out", out, shape, n, (_BF16,), index),
          _status_ptr(status, index), _stream_of(stream, index))
    return out


def expert_swiglu(x, x_scales, w13, w13_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None, expected_rows=0):
    """silu(x wg^T) * (x wu^T) per expert, w13 = [gate; up] [E][2I][K], requantised:
    (codes [rows][I] uint8, scales [rows][I / 128]) (or [E][cap][..])."""
    index, shape, n, cx, cg, cw = _products("expert_swiglu", x, x_scales, w13, w13_scales, counts, offsets, bases, expected_rows)
    if n % 256:
        _refuse(f"expert_swiglu: {n} weight rows are no gate and up of a multiple of 128 each")
    inter = n // 2
    if out is None:
        out = _empty(x, stream, (*shape[:-1], inter), _U8), _empty(x, stream, (*shape[:-1], inter // 128), _F32)
    codes, scales = out
    _call("ep_expert_swiglu", index, cx, cg, cw, codes.data_ptr(),
          _output("expert_swiglu: out codes", codes, shape, inter, _CODES, index), scales.data_ptr(),
          _output("expert_swiglu: out scales", scales, shape, inter // 128, (_F32,), index), _status_ptr(status, index),
          _stream_of(stream, index))
    return codes, scales


def moe_tokens(x, topk_idx, topk_weights, w13, w2, w13_scales=None, w2_scales=None, out=None, workspace=None, status=None,
               stream=None):
    """The whole layer for up to 64 tokens, without dispatch and combine:
    out[t] = sum_k topk_weights[t][k] * W2[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])), e = topk_idx[t][k], -1 skipped.

    x [T][H] bf16; w13 = [gate; up] [E][2I][H] and w2 [E][H][I], bf16, or e4m3 codes with their block scales.
    `workspace` (contiguous, moe_tokens_workspace bytes) is allocated when it is not given."""
    index = x.get_device()
    xs, ts, ws, vs = x.shape, topk_idx.shape, w13.shape, w2.shape
    if index < 0:
        _refuse("moe_tokens: all tensors must be on a CUDA device")
    if x.dtype != _BF16 or len(xs) != 2:
        _refuse(f"moe_tokens: x bf16 [T][H]: got {x.dtype} {tuple(xs)}")
    T, H = xs
    if topk_idx.dtype != torch.int64 or len(ts) != 2 or ts[0] != T or not topk_idx.is_contiguous():
        _refuse(f"moe_tokens: topk_idx int64 [{T}][K], contiguous: got {topk_idx.dtype} {tuple(ts)}")
    if topk_weights.dtype != _F32 or topk_weights.shape != ts or not topk_weights.is_contiguous():
        _refuse(f"moe_tokens: topk_weights fp32 {tuple(ts)}, contiguous: got {topk_weights.dtype} {tuple(topk_weights.shape)}")
    K = ts[1]
    if len(ws) != 3 or len(vs) != 3 or not w13.is_contiguous() or not w2.is_contiguous():
        _refuse("moe_tokens: weights [E][rows][cols], contiguous")
    E, I = ws[0], vs[2]
    if ws[1] != 2 * I or ws[2] != H or vs[0] != E or vs[1] != H:
        _refuse(f"moe_tokens: w13 {tuple(ws)}, w2 {tuple(vs)} for {H} channels")
    p13 = p2 = 0
    if w13_scales is None and w2_scales is None:
        if w13.dtype != _BF16 or w2.dtype != _BF16:
            _refuse(f"moe_tokens: weights without scales are bf16: got {w13.dtype}, {w2.dtype}")
    else:
        if w13_scales is None or w2_scales is None or w13.dtype not in _CODES or w2.dtype not in _CODES:
            _refuse("moe_tokens: e4m3 codes with scales for both weights, or bf16 without")
        for t, r, c in ((w13_scales, 2 * I, H), (w2_scales, H, I)):
            if t.dtype != _F32 or t.shape != (E, r // 128, c // 128) or not t.is_contiguous() or t.get_device() != index:
                _refuse(f"moe_tokens: weight scales fp32 {(E, r // 128, c // 128)}, contiguous, on the same device")
        p13, p2 = w13_scales.data_ptr(), w2_scales.data_ptr()
    if (topk_idx.get_device() != index or topk_weights.get_device() != index or w13.get_device() != index
            or w2.get_device() != index or (workspace is not None and workspace.get_device() != index)):
        _refuse("moe_tokens: all tensors must be on the same CUDA device")
    if out is None:
        out = _empty(x, stream, (T, H), _BF16)
    if workspace is None:
        workspace = _empty(x, stream, (_workspace_bytes(index, T, K, E, H, I, p13 != 0),), _U8)
    elif not workspace.is_contiguous():
        _refuse(f"moe_tokens: workspace must be contiguous (strides {workspace.stride()})")
    _call("ep_moe_tokens", index, x.data_ptr(), _step("moe_tokens", x), T, topk_idx.data_ptr(), topk_weights.data_ptr(), K,
          _MOE(w13.data_ptr(), p13, w2.data_ptr(), p2, E, H, I), out.data_ptr(),
          _output("moe_tokens: out", out, xs, H, (_BF16,), index), workspace.data_ptr(), workspace.nbytes,
          _status_ptr(status, index), _stream_of(stream, index))
    return out


def moe_tokens_workspace(num_tokens: int, num_topk: int, experts: int, hidden: int, inter: int, fp8: bool = True) -> int:
    """Bytes of workspace moe_tokens needs on the current device (0 for sizes it refuses)."""
    return int(_lib.load().ep_moe_tokens_workspace(num_tokens, num_topk, _MOE(0, int(fp8), 0, int(fp8), experts, hidden, inter)))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index: int, *sizes) -> int:
    with torch.cuda.device(index):
        return moe_tokens_workspace(*sizes)
