"""MoELayer with bf16 weights, which have no scales: the few-token form, as before MXFP4 weights came in."""
import pytest
import torch

from combine_get_dispatch_histograms_gb300 import Context, inputs, moe_tokens
from combine_get_dispatch_histograms_gb300.layer import MoELayer
from expert_util import gen, randn

BF = torch.bfloat16


def test_weights_without_scales_are_no_mxfp4():
    w = torch.zeros(1, dtype=BF)
    layer = MoELayer(w, None, w, None)
    assert not layer.fp4
    with pytest.raises(ValueError, match="up to 64 tokens"):
        layer.forward_ll(None, None, None, None)
    with pytest.raises(ValueError, match="both"):
        MoELayer(w, torch.zeros(1, dtype=torch.uint8), w, None)


@pytest.mark.gpu
def test_few_tokens_of_bf16_weights():
    R, E, K, T, H, I = 4, 8, 2, 16, 128, 256
    g = gen(3)
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    w13, w2 = (randn((E, 2 * I, H), g) * H ** -0.5).to(BF), (randn((E, H, I), g) * I ** -0.5).to(BF)
    ctx = Context(R, E, K, T, H)
    out = MoELayer(w13, None, w2, None).forward(ctx, x, idx, v)
    ctx.check()
    assert torch.equal(out.view(-1, H), moe_tokens(x.view(-1, H), idx.view(-1, K), v.view(-1, K), w13, w2))
    more = Context(R, E, K, T + 1, H)
    with pytest.raises(ValueError, match="up to 64 tokens"):
        MoELayer(w13, None, w2, None).forward(more, x, idx, v)
