"""A mixture-of-experts layer over the dispatch path: three ways to run the same weights.

    layer = MoELayer(w13, w13_scales, w2, w2_scales)
    out = layer.forward(ctx, x, topk_idx, topk_weights)         # x [R][T][H] bf16 over a Context
    out = layer.forward_ll(buf, x, topk_idx, topk_weights)      # over a low-latency LLBuffer

forward chooses by the number of tokens in all: up to FEW_TOKENS run as
moe_tokens (two to four kernels, x in bf16); more are quantised and dispatched
into the per-expert blocks, run through the two expert products and combined.
Neither form waits on the host, so each can be captured in a CUDA graph.
"""
from __future__ import annotations

import torch

from . import Context, LLBuffer, moe_tokens

# The most tokens moe_tokens takes.
FEW_TOKENS = 64


class MoELayer:
    """w13 = [gate; up] [E][2I][H] and w2 [E][H][I]: e4m3 codes with scales per 128 x 128 block."""

    def __init__(self, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor, w2_scales: torch.Tensor):
        self.w13, self.w13_scales, self.w2, self.w2_scales = w13, w13_scales, w2, w2_scales

    def forward(self, ctx: Context, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor) -> torch.Tensor:
        """x, out [R][T][H] bf16; topk_idx, topk_weights [R][T][K].  Device errors: ctx.check()."""
        if ctx.R * ctx.T <= FEW_TOKENS:
            return moe_tokens(x.view(-1, ctx.H), topk_idx.view(-1, ctx.K), topk_weights.view(-1, ctx.K), self.w13, self.w2,
                              self.w13_scales, self.w2_scales, status=ctx.lib.ep_ctx_status_word(ctx._ctx)).view(x.shape)
        _, h = ctx.layout_notify(topk_idx, wait=False)
        rows = ctx.dispatch_permuted_quant(x, topk_idx, topk_weights, h)["permuted_xq"]
        hidden = ctx.expert_swiglu(h, rows, self.w13, self.w13_scales)
        return ctx.combine(h, ctx.expert_gemm(h, hidden, self.w2, self.w2_scales), topk_idx, topk_weights)

    def forward_ll(self, buf: LLBuffer, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor) -> torch.Tensor:
        """The same through the low-latency buffer (T <= cap tokens per rank).  Device errors: buf.check()."""
        packed = buf.dispatch(x, topk_idx)
        hidden = buf.expert_swiglu(packed, self.w13, self.w13_scales)
        return buf.combine(buf.expert_gemm(hidden, packed, self.w2, self.w2_scales), topk_idx, topk_weights, packed)
