"""The router before dispatch: the choice of experts, the balance loss with its counts, and the gradient of the logits.

    topk_idx, topk_weights = route(logits, 8)                          # what dispatch, combine and moe_tokens take
    got = balance_loss(logits, topk_idx, coef=0.01)                    # got["loss"], got["counts"], got["factors"]
    dlogits = router_backward(logits, topk_idx, dweights, factors=got["factors"], dloss=dloss)

logits are fp32 or bf16 [T][E] or [R][T][E] (rows evenly spaced), E up to 1024 and the choices up to 32; topk_idx int64
and topk_weights fp32 have the same leading dimensions.  Context.route takes the sizes of its context.
"""
from __future__ import annotations

import struct

import torch

from . import _lib
from .experts import _call, _empty, _refuse, _status_ptr, _step, _stream_of
from .norm import _workspace_bytes

_I64, _I32, _F32, _U8, _BOOL = torch.int64, torch.int32, torch.float32, torch.uint8, torch.bool
_TYPES = {torch.bfloat16: 0, _F32: 1}
_SCORING = {"softmax": 0, "sigmoid": 1}
_KEYS = {"logits": 0, "scores": 1}
_PACK = struct.Struct("@qiiiiiiifii0P").pack   # ep_router as the C side lays it out


def _ROUTER(tokens, experts, topk, logits_type, scoring, normalize, groups, topk_groups, scale, keys=0, group_keys=2):
    return _PACK(tokens, experts, topk, logits_type, scoring, normalize, groups, topk_groups, scale, keys, group_keys)


def _logits(name, t):
    """(device index, shape, elements between rows)."""
    index, shape = t.get_device(), t.shape
    if index < 0:
        _refuse(f"{name}: all tensors must be on a CUDA device")
    if t.dtype not in _TYPES or len(shape) not in (2, 3) or shape[-1] == 0:
        _refuse(f"{name}: fp32 or bf16 [T][E] or [R][T][E]: got {t.dtype} {tuple(shape)}")
    return index, shape, _step(name, t)


def _plain(name, t, shape, dtype, index):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        _refuse(f"{name}: {dtype} {tuple(shape)}, contiguous, on the same CUDA device: got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _descriptor(name, logits, shape, topk, scoring, normalize=True, groups=1, topk_groups=1, scale=1.0, keys="logits",
                group_keys=2):
    if scoring not in _SCORING:
        _refuse(f"{name}: scoring {scoring!r}: 'softmax' or 'sigmoid'")
    if keys not in _KEYS or group_keys not in (1, 2):
        _refuse(f"{name}: keys {keys!r}: 'logits' or 'scores'; group_keys {group_keys!r}: 1 or 2")
    tokens = shape[0] * (shape[1] if len(shape) == 3 else 1)
    return _ROUTER(tokens, shape[-1], topk, _TYPES[logits.dtype], _SCORING[scoring], bool(normalize), groups, topk_groups, scale, _KEYS[keys],
                   group_keys)


def route(logits, topk: int, bias=None, mask=None, scoring="softmax", normalize=True, scale=1.0, groups=1, topk_groups=None, out=None,
          stream=None, *, keys="logits", group_keys=2):
    """(topk_idx int64, topk_weights fp32) [..][topk]: the experts with the largest key, the lowest of equal ones first, and
    their weights from the logits alone.

    scoring "softmax": over all experts, or with normalize over the chosen; "sigmoid": with normalize over the chosen
    ones' sum + 1e-20; all times scale.  -inf is never chosen: entries without an expert are -1 with weight 0.
    bias fp32 [E]; mask [..] (bool or uint8), 0 for padding.
    keys "logits": key = logit + bias; "scores": key = score + bias, the score by `scoring` (the softmax over all experts),
    as a router is trained whose bias balances the load.  The two choose differently where there is a bias or where groups
    are ranked by sums.
    groups, topk_groups: choose among the experts of the topk_groups of `groups` equal runs of experts (the experts of a
    node, say) with the largest sum of their two largest keys, or with group_keys=1 the largest key."""
    index, shape, step = _logits("route: logits", logits)
    lead = shape[:-1]
    r = _descriptor("route", logits, shape, topk, scoring, normalize, groups, groups if topk_groups is None else topk_groups, scale, keys,
                    group_keys)
    bias_at = None if bias is None else _plain("route: bias", bias, shape[-1:], _F32, index)
    mask_at = None if mask is None else _plain("route: mask", mask, lead, _BOOL if mask.dtype == _BOOL else _U8, index)
    shape = (*lead, topk)
    if out is None:
        idx, weights = _empty(logits, stream, shape, _I64), _empty(logits, stream, shape, _F32)
    else:
        idx, weights = out
        _plain("route: out topk_idx", idx, shape, _I64, index)
        _plain("route: out topk_weights", weights, shape, _F32, index)
    _call("ep_route", index, r, logits.data_ptr(), step, bias_at, mask_at, idx.data_ptr(), weights.data_ptr(), _stream_of(stream, index))
    return idx, weights


def balance_loss(logits, topk_idx, coef=1.0, scoring="softmax", out=None, workspace=None, status=None, stream=None) -> dict:
    """{"loss": fp32 [1], "counts": int32 [S][E], "factors": fp32 [S][E]} over the S sequences of logits [S][T][E] (or one, [T][E]):
    loss = coef * the sequences' mean of sum_e E * (share of the choices that name e) * (mean of e's score over the tokens).

    Scores are the softmax, or the sigmoids over their sum.  -1 entries and tokens without an entry count for nothing.
    factors are what router_backward takes.  out: a dict with the three to write into; `workspace` (contiguous,
    balance_loss_workspace bytes) is allocated when it is not given; status as for moe_tokens."""
    index, shape, step = _logits("balance_loss: logits", logits)
    lead, experts = shape[:-1], shape[-1]
    if topk_idx.dim() != len(shape):
        _refuse(f"balance_loss: topk_idx int64 {tuple(lead)}[K]: got {tuple(topk_idx.shape)}")
    topk = topk_idx.shape[-1]
    sequences = lead[0] if len(lead) == 2 else 1
    idx_at = _plain("balance_loss: topk_idx", topk_idx, (*lead, topk), _I64, index)
    r = _descriptor("balance_loss", logits, shape, topk, scoring)
    if out is None:
        shape = (sequences, experts)
        loss, counts, factors = _empty(logits, stream, (1,), _F32), _empty(logits, stream, shape, _I32), _empty(logits, stream, shape, _F32)
    else:
        loss, counts, factors = out["loss"], out["counts"], out["factors"]
        _plain("balance_loss: out loss", loss, (1,), _F32, index)
        _plain("balance_loss: out counts", counts, (sequences, experts), _I32, index)
        _plain("balance_loss: out factors", factors, (sequences, experts), _F32, index)
    if workspace is None:
        workspace = _empty(logits, stream, (_workspace_bytes("ep_balance_loss_workspace", index, r, sequences),), _U8)
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        _refuse("balance_loss: workspace must be contiguous, on the same device")
    _call("ep_balance_loss", index, r, logits.data_ptr(), step, idx_at, sequences, coef, loss.data_ptr(), counts.data_ptr(),
          factors.data_ptr(), workspace.data_ptr(), workspace.nbytes, _status_ptr(status, index), _stream_of(stream, index))
    return {"loss": loss, "counts": counts, "factors": factors}


def balance_loss_workspace(tokens: int, experts: int, sequences: int = 1) -> int:
    """Bytes of workspace balance_loss needs on the current device for this many tokens in all (0 for sizes it refuses)."""
    return int(_lib.load().ep_balance_loss_workspace(_ROUTER(tokens, experts, 1, 0, 0, 1, 1, 1, 1.0), sequences))


def router_backward(logits, topk_idx, dweights=None, factors=None, dloss=None, scoring="softmax", normalize=True, scale=1.0, out=None,
                    status=None, stream=None):
    """The logits' gradient, of their type: of route's weights, given dweights fp32 [..][topk], and of balance_loss, given its
    factors and dloss fp32 [1].  scoring, normalize and scale as they were; the choice and the factors are constants.
    out may be the logits themselves."""
    index, shape, step = _logits("router_backward: logits", logits)
    lead, experts = shape[:-1], shape[-1]
    if topk_idx.dim() != len(shape):
        _refuse(f"router_backward: topk_idx int64 {tuple(lead)}[K]: got {tuple(topk_idx.shape)}")
    topk = topk_idx.shape[-1]
    sequences = lead[0] if len(lead) == 2 else 1
    idx_at = _plain("router_backward: topk_idx", topk_idx, (*lead, topk), _I64, index)
    dw_at = None if dweights is None else _plain("router_backward: dweights", dweights, (*lead, topk), _F32, index)
    f_at = None if factors is None else _plain("router_backward: factors", factors, (sequences, experts), _F32, index)
    dl_at = None if dloss is None else _plain("router_backward: dloss", dloss, (1,), _F32, index)
    r = _descriptor("router_backward", logits, shape, topk, scoring, normalize, 1, 1, scale)
    out_step = experts
    if out is None:
        out = _empty(logits, stream, shape, logits.dtype)
    elif out.dtype != logits.dtype or out.shape != shape or out.get_device() != index:
        _refuse(f"router_backward: out {logits.dtype} {tuple(shape)} on the same CUDA device: got {out.dtype} {tuple(out.shape)}")
    else:
        out_step = _step("router_backward: out", out)
    _call("ep_router_backward", index, r, logits.data_ptr(), step, idx_at, dw_at, f_at, sequences, dl_at, out.data_ptr(), out_step,
          _status_ptr(status, index), _stream_of(stream, index))
    return out
