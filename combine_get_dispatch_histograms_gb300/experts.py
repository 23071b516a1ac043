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

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import EpError, EpFp8Rows, EpFp8Weight, EpMoeWeights, EpRowGroups, check

_CODES = (torch.uint8, torch.float8_e4m3fn)
# bits of a status word, as the C entry points OR them in, by the status a check raises first
_STATUS_BITS = ((1, -2, "topk_idx holds a value outside [-1, E)"), (4, -4, "a bounded device wait ran out"),
                (2, -3, "a group's rows lie outside the row arrays"))


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


def _stream_of(stream, device):
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _need(ok: bool, text: str):
    if not ok:
        raise ValueError(text)


def _on(device, **ts):
    for name, t in ts.items():
        if t is not None:
            _need(t.is_cuda and t.device == device, f"{name} must be on {device}")


def _codes_scales(name: str, codes: torch.Tensor, scales: torch.Tensor):
    """Codes [..][K] and scales [..][K / 128] of rows that are evenly spaced: (rows, K, strides)."""
    _need(codes.dtype in _CODES and codes.dim() in (2, 3), f"{name}: codes [rows][K] or [E][rows][K], uint8 or e4m3")
    _need(scales.dtype == torch.float32 and scales.dim() == codes.dim(), f"{name}: fp32 scales of the codes' rank")
    k = codes.shape[-1]
    _need(k > 0 and k % 128 == 0, f"{name}: {k} channels are no multiple of 128")
    _need(tuple(scales.shape) == (*codes.shape[:-1], k // 128),
          f"{name}: scales {tuple(scales.shape)} for codes {tuple(codes.shape)}")
    rows = codes.numel() // k
    strides = []
    for t in (codes, scales):
        step = t.stride(-2) if t.shape[-2] > 1 else (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else t.shape[-1])
        _need(t.shape[-1] == 1 or t.stride(-1) == 1, f"{name}: channels must be contiguous")
        _need(t.dim() == 2 or t.shape[0] <= 1 or t.stride(0) == t.shape[1] * step, f"{name}: regions must be evenly spaced")
        strides.append(step if rows > 1 else max(step, t.shape[-1]))
    return rows, k, strides[0], strides[1]


class _Call:
    """The C descriptors of one product, checked."""

    def __init__(self, name, x, x_scales, w, w_scales, counts, offsets, bases=None):
        dev = x.device
        _need(x.is_cuda, f"{name}: all tensors must be on a CUDA device")
        _on(dev, x_scales=x_scales, w=w, w_scales=w_scales, counts=counts, offsets=offsets, bases=bases)
        self.device = dev
        self.rows, k, cs, ss = _codes_scales(name, x, x_scales)
        _need(w.dtype in _CODES and w.dim() in (2, 3) and w.is_contiguous(), f"{name}: weight codes [E][N][K] or [N][K], contiguous")
        groups = w.shape[0] if w.dim() == 3 else 1
        n = w.shape[-2]
        _need(w.shape[-1] == k, f"{name}: weight of {w.shape[-1]} channels for rows of {k}")
        want = (groups, (n + 127) // 128, k // 128) if w.dim() == 3 else ((n + 127) // 128, k // 128)
        _need(w_scales.dtype == torch.float32 and tuple(w_scales.shape) == want and w_scales.is_contiguous(),
              f"{name}: weight scales fp32 {want}, contiguous")
        for what, t in (("counts", counts), ("offsets", offsets)):
            _need(t is None or (t.dtype == torch.int32 and t.numel() == groups and t.is_contiguous()),
                  f"{name}: {what} int32 [{groups}], contiguous")
        if x.dim() == 3:
            _need(x.shape[0] == groups, f"{name}: {x.shape[0]} regions for {groups} groups")
            _need(offsets is None, f"{name}: regions take no offsets")
            stride = x.shape[1]
        else:
            _need(groups == 1 or (counts is not None and offsets is not None), f"{name}: {groups} groups need counts and offsets")
            stride = self.rows
        per_base = 0
        if bases is not None:
            _need(bases.dtype == torch.int32 and bases.is_contiguous(), f"{name}: bases int32")
            per_base = groups // max(1, bases.numel() - 1)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.n, self.lead = n, tuple(x.shape[:-1])
        self.x = EpFp8Rows(x.data_ptr(), cs, x_scales.data_ptr(), ss, self.rows)
        self.g = EpRowGroups(p(counts), p(offsets), p(bases), per_base, stride)
        self.w = EpFp8Weight(w.data_ptr(), w_scales.data_ptr(), groups, n, k)

    def run(self, fn, stream, *args):
        lib = _lib.load()
        with torch.cuda.device(self.device):
            check(fn, getattr(lib, fn)(ctypes.byref(self.x), ctypes.byref(self.g), ctypes.byref(self.w), *args,
                                       _stream_of(stream, self.device)))


def fp8_row_views(rows: torch.Tensor, channels: int):
    """(codes, scales) of FP8 rows [rows][row bytes]: `channels` e4m3 codes, then channels / 128 fp32 scales."""
    return rows[:, :channels], rows[:, channels:channels + channels // 32].view(torch.float32)


def _status_ptr(status, device):
    if status is None or isinstance(status, int):  # an address: the status word of a context or a buffer
        return status
    _need(status.dtype in (torch.int32, torch.uint32) and status.numel() >= 1, "status: an int32 device word")
    _on(device, status=status)
    return status.data_ptr()


def _row_stride(name, t, lead, n):
    """Elements between the rows of an output [..lead][n] whose rows are evenly spaced."""
    _need(tuple(t.shape) == (*lead, n), f"{name}: shape {tuple(t.shape)}, expected {(*lead, n)}")
    rows = t.numel() // max(1, n)
    step = t.stride(-2) if t.shape[-2] > 1 else (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else n)
    _need(n == 1 or t.stride(-1) == 1, f"{name}: channels must be contiguous")
    _need(t.dim() == 2 or t.shape[0] <= 1 or t.stride(0) == t.shape[1] * step, f"{name}: regions must be evenly spaced")
    return step if rows > 1 else max(step, n)


def expert_gemm(x, x_scales, w, w_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None):
    """y = x w^T per expert: bf16 [rows][N] (or [E][cap][N]).  Rows of no expert are not written."""
    c = _Call("expert_gemm", x, x_scales, w, w_scales, counts, offsets, bases)
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.empty(*c.lead, c.n, dtype=torch.bfloat16, device=c.device)
    _on(c.device, out=out)
    _need(out.dtype == torch.bfloat16, "expert_gemm: out is bf16")
    c.run("ep_expert_gemm", stream, out.data_ptr(), _row_stride("expert_gemm: out", out, c.lead, c.n), _status_ptr(status, c.device))
    return out


def expert_swiglu(x, x_scales, w13, w13_scales, counts=None, offsets=None, out=None, status=None, stream=None, *, bases=None):
    """silu(x wg^T) * (x wu^T) per expert, w13 = [gate; up] [E][2I][K], requantised:
    (codes [rows][I] uint8, scales [rows][I / 128]) (or [E][cap][..])."""
    c = _Call("expert_swiglu", x, x_scales, w13, w13_scales, counts, offsets, bases)
    _need(c.n % 256 == 0, f"expert_swiglu: {c.n} weight rows are no gate and up of a multiple of 128 each")
    inter = c.n // 2
    if out is None:
        with torch.cuda.stream(stream):
            out = (torch.empty(*c.lead, inter, dtype=torch.uint8, device=c.device),
                   torch.empty(*c.lead, inter // 128, dtype=torch.float32, device=c.device))
    codes, scales = out
    _on(c.device, out=codes, out_scales=scales)
    _need(codes.dtype in _CODES and scales.dtype == torch.float32, "expert_swiglu: out is (codes, fp32 scales)")
    c.run("ep_expert_swiglu", stream, codes.data_ptr(), _row_stride("expert_swiglu: out codes", codes, c.lead, inter),
          scales.data_ptr(), _row_stride("expert_swiglu: out scales", scales, c.lead, inter // 128), _status_ptr(status, c.device))
    return codes, scales


def moe_tokens(x, topk_idx, topk_weights, w13, w2, w13_scales=None, w2_scales=None, out=None, workspace=None, status=None,
               stream=None):
    """The whole layer for up to 64 tokens, without dispatch and combine:
    out[t] = sum_k topk_weights[t][k] * W2[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])), e = topk_idx[t][k], -1 skipped.

    x [T][H] bf16; w13 = [gate; up] [E][2I][H] and w2 [E][H][I], bf16, or e4m3 codes with their block scales.
    `workspace` (uint8, moe_tokens_workspace bytes) is allocated when it is not given."""
    _need(x.is_cuda, "moe_tokens: all tensors must be on a CUDA device")
    dev = x.device
    _on(dev, topk_idx=topk_idx, topk_weights=topk_weights, w13=w13, w2=w2, w13_scales=w13_scales, w2_scales=w2_scales, out=out,
        workspace=workspace)
    _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1, "moe_tokens: x bf16 [T][H], channels contiguous")
    T, H = x.shape
    _need(topk_idx.dim() == 2 and topk_idx.shape[0] == T and topk_idx.dtype == torch.int64 and topk_idx.is_contiguous(),
          "moe_tokens: topk_idx int64 [T][K], contiguous")
    _need(topk_weights.shape == topk_idx.shape and topk_weights.dtype == torch.float32 and topk_weights.is_contiguous(),
          "moe_tokens: topk_weights fp32 of topk_idx's shape, contiguous")
    K = topk_idx.shape[1]
    _need(w13.dim() == 3 and w2.dim() == 3 and w13.is_contiguous() and w2.is_contiguous(), "moe_tokens: weights [E][rows][cols], contiguous")
    E, I = w13.shape[0], w2.shape[2]
    _need(tuple(w13.shape) == (E, 2 * I, H) and tuple(w2.shape) == (E, H, I),
          f"moe_tokens: w13 {tuple(w13.shape)}, w2 {tuple(w2.shape)} for {H} channels")
    fp8 = w13_scales is not None or w2_scales is not None
    if fp8:
        _need(w13_scales is not None and w2_scales is not None, "moe_tokens: scales for both weights, or for none")
        _need(w13.dtype in _CODES and w2.dtype in _CODES, "moe_tokens: weights with scales are e4m3 codes")
        for name, t, r, c in (("w13_scales", w13_scales, 2 * I, H), ("w2_scales", w2_scales, H, I)):
            _need(t.dtype == torch.float32 and t.is_contiguous() and tuple(t.shape) == (E, r // 128, c // 128),
                  f"moe_tokens: {name} fp32 {(E, r // 128, c // 128)}, contiguous")
    else:
        _need(w13.dtype == w2.dtype == torch.bfloat16, "moe_tokens: weights without scales are bf16")
    lib = _lib.load()
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        if out is None:
            out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        if workspace is None:
            workspace = torch.empty(int(lib.ep_moe_tokens_workspace(T, K, H, I)), dtype=torch.uint8, device=dev)
        _need(out.dtype == torch.bfloat16, "moe_tokens: out is bf16")
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        w = EpMoeWeights(w13.data_ptr(), p(w13_scales), w2.data_ptr(), p(w2_scales), E, H, I)
        check("ep_moe_tokens", lib.ep_moe_tokens(
            x.data_ptr(), x.stride(0) if T > 1 else H, T, topk_idx.data_ptr(), topk_weights.data_ptr(), K, ctypes.byref(w),
            out.data_ptr(), _row_stride("moe_tokens: out", out, (T,), H), workspace.data_ptr(), workspace.numel(),
            _status_ptr(status, dev), _stream_of(stream, dev)))
    return out


def moe_tokens_workspace(num_tokens: int, num_topk: int, hidden: int, inter: int) -> int:
    """Bytes of workspace moe_tokens needs (0 for sizes it refuses)."""
    return int(_lib.load().ep_moe_tokens_workspace(num_tokens, num_topk, hidden, inter))
