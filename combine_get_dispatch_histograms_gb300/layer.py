"""A mixture-of-experts layer over the dispatch path: three ways to run the same weights.

    layer = MoELayer(w13, w13_scales, w2, w2_scales)
    out = layer.forward(ctx, x, topk_idx, topk_weights)         # x [R][T][H] bf16 over a Context
    out = layer.forward_ll(buf, x, topk_idx, topk_weights)      # over a low-latency LLBuffer

forward chooses by the number of tokens in all: up to FEW_TOKENS run as
moe_tokens (two to four kernels, x in bf16); more are quantised and dispatched
into the per-expert blocks, run through the two expert products and combined.
Neither form waits on the host, so each can be captured in a CUDA graph.

With MXFP4 weights (scales in uint8) forward always dispatches, rows of 4 bits.
"""
from __future__ import annotations

import torch

from . import Context, LLBuffer, moe_tokens

# The most tokens moe_tokens takes.
FEW_TOKENS = 64


class MoELayer:
    """w13 = [gate; up] [E][2I][H] and w2 [E][H][I]: e4m3 codes with fp32 scales per 128 x 128 block, or MXFP4 codes
    [..][H/2], [..][I/2] with uint8 scales [..][H/32], [..][I/32].  bf16 weights, without scales (None), run up to FEW_TOKENS
    tokens."""

    def __init__(self, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor, w2_scales: torch.Tensor):
        self.w13, self.w13_scales, self.w2, self.w2_scales = w13, w13_scales, w2, w2_scales
        four = [s is not None and s.dtype == torch.uint8 for s in (w13_scales, w2_scales)]
        self.fp4 = four[0]
        if four[0] != four[1]:
            raise ValueError("MoELayer: both weights e4m3 with fp32 scales, or both MXFP4 with uint8 scales")

    def forward(self, ctx: Context, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor) -> torch.Tensor:
        """x, out [R][T][H] bf16; topk_idx, topk_weights [R][T][K].  Device errors: ctx.check()."""
        if self.fp4:
            _, h = ctx.layout_notify(topk_idx, wait=False)
            rows = ctx.dispatch_permuted_fp4(ctx.quantize_fp4(x), topk_idx, topk_weights, h)["permuted_xq"]
            hidden = ctx.expert_swiglu_fp4(h, rows, self.w13, self.w13_scales)
            return ctx.combine(h, ctx.expert_gemm_fp4(h, hidden, self.w2, self.w2_scales), topk_idx, topk_weights)
        if ctx.R * ctx.T <= FEW_TOKENS:
            return moe_tokens(x.view(-1, ctx.H), topk_idx.view(-1, ctx.K), topk_weights.view(-1, ctx.K), self.w13, self.w2,
                              self.w13_scales, self.w2_scales, status=ctx.lib.ep_ctx_status_word(ctx._ctx)).view(x.shape)
        self._need_scales("forward")
        _, h = ctx.layout_notify(topk_idx, wait=False)
        rows = ctx.dispatch_permuted_quant(x, topk_idx, topk_weights, h)["permuted_xq"]
        hidden = ctx.expert_swiglu(h, rows, self.w13, self.w13_scales)
        return ctx.combine(h, ctx.expert_gemm(h, hidden, self.w2, self.w2_scales), topk_idx, topk_weights)

    def forward_ll(self, buf: LLBuffer, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor) -> torch.Tensor:
        """The same through the low-latency buffer (T <= cap tokens per rank; e4m3 weights, as its messages).  Device
        errors: buf.check()."""
        if self.fp4:
            raise ValueError("MoELayer.forward_ll: the low-latency buffer carries FP8 rows, for e4m3 weights")
        self._need_scales("forward_ll")
        packed = buf.dispatch(x, topk_idx)
        hidden = buf.expert_swiglu(packed, self.w13, self.w13_scales)
        return buf.combine(buf.expert_gemm(hidden, packed, self.w2, self.w2_scales), topk_idx, topk_weights, packed)

    def _need_scales(self, name: str):
        if self.w13_scales is None or self.w2_scales is None:
            raise ValueError(f"MoELayer.{name}: weights without scales run up to {FEW_TOKENS} tokens, by forward")
