"""The experts between dispatch and combine: MoELayer's three forms against a 64-bit layer.

The forms that dispatch FP8 rows round x and h to e4m3 (relative step 2^-3, so an error of at most 2^-4 and 2^-4 / sqrt(3)
= 0.036 in the mean square); x's errors reach both factors of h, so the output's relative 2-norm is off by about
sqrt(3) * 0.036 = 0.06, held to 0.12.  A wrong row, expert, scale or weight is off by about 1."""
import pytest
import torch

from combine_get_dispatch_histograms_gb300 import Context, LLBuffer, inputs
from combine_get_dispatch_histograms_gb300.layer import MoELayer
from expert_util import gen, quantize_weight, randn, silu64, weight64

gpu = pytest.mark.gpu


def layer_and_reference(E, H, I, x, idx, v, seed):
    g = gen(seed)
    w13, s13 = quantize_weight(randn((E, 2 * I, H), g) * H ** -0.5)
    w2, s2 = quantize_weight(randn((E, H, I), g) * I ** -0.5)
    X, J, V = x.view(-1, H).double(), idx.view(-1, idx.shape[-1]), v.view(-1, idx.shape[-1]).double()
    ref = torch.zeros_like(X)
    for e in range(E):
        t, k = torch.nonzero(J == e, as_tuple=True)
        y = X[t] @ weight64(w13[e], s13[e]).t()
        h = silu64(y[:, :I]) * y[:, I:]
        ref.index_add_(0, t, V[t, k][:, None] * (h @ weight64(w2[e], s2[e]).t()))
    return MoELayer(w13, s13, w2, s2), ref.view(x.shape)


def far(out, ref):
    return float((out.double() - ref).norm() / ref.norm())


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I,align", [(4, 8, 2, 40, 128, 128, 1), (2, 16, 4, 300, 512, 384, 1), (4, 12, 3, 65, 256, 640, 16)])
def test_forward_over_dispatch(R, E, K, T, H, I, align):
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    layer, ref = layer_and_reference(E, H, I, x, idx, v, 4)
    ctx = Context(R, E, K, T, H, expert_alignment=align)
    out = layer.forward(ctx, x, idx, v)
    ctx.check()
    assert far(out, ref) < 0.12
    h = ctx.notify_dispatch(idx, ctx.get_dispatch_layout(idx))   # the waiting form gives the same
    rows = ctx.dispatch_permuted_quant(x, idx, v, h)["permuted_xq"]
    y = ctx.expert_gemm(h, ctx.expert_swiglu(h, rows, layer.w13, layer.w13_scales), layer.w2, layer.w2_scales)
    assert torch.equal(ctx.combine(h, y, idx, v).view(torch.int16), out.view(torch.int16))


@gpu
def test_forward_of_few_tokens():
    R, E, K, T, H, I = 4, 8, 2, 16, 128, 256
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    layer, ref = layer_and_reference(E, H, I, x, idx, v, 5)
    ctx = Context(R, E, K, T, H)
    out = layer.forward(ctx, x, idx, v)
    ctx.check()
    assert far(out, ref) < 4e-3                                   # bf16 rounding alone


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I", [(4, 8, 2, 16, 128, 128), (2, 16, 4, 100, 512, 256)])
def test_forward_low_latency(R, E, K, T, H, I):
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    layer, ref = layer_and_reference(E, H, I, x, idx, v, 6)
    buf = LLBuffer(R, E, K, T, H, T)
    out = layer.forward_ll(buf, x, idx, v)
    buf.check()
    assert far(out, ref) < 0.12


@gpu
def test_forward_in_a_graph_on_new_routing():
    R, E, K, T, H, I = 2, 16, 4, 100, 256, 128
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3).cuda()
    ctx = Context(R, E, K, T, H)
    layer, _ = layer_and_reference(E, H, I, x, idx, v, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(ctx, x, idx, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(ctx, x, idx, v)
    idx.copy_(inputs.random_topk(R, E, K, T, 9, mask_p=0.5).cuda())
    graph.replay()
    ctx.check()
    _, ref = layer_and_reference(E, H, I, x, idx, v, 7)
    assert far(out, ref) < 0.12


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I", [(4, 8, 2, 40, 256, 128), (2, 6, 2, 20, 256, 128)])
def test_a_tokens_nan_stays_a_nan(R, E, K, T, H, I):
    """Over dispatch, over the low-latency buffer and (40 tokens) as a few-token layer: no finite output for it."""
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3).cuda()
    layer, _ = layer_and_reference(E, H, I, x, idx, v, 8)
    x[1, 3, 17] = x[0, 5, H - 1] = float("nan")
    ctx, buf = Context(R, E, K, T, H), LLBuffer(R, E, K, T, H, T)
    for out in (layer.forward(ctx, x, idx, v), layer.forward_ll(buf, x, idx, v)):
        bad = torch.zeros(R, T, dtype=torch.bool, device="cuda")
        bad[1, 3] = bad[0, 5] = True
        assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    ctx.check()
    buf.check()


@gpu
def test_a_token_of_nothing_but_nan_stays_a_nan():
    R, E, K, T, H, I = 4, 8, 2, 40, 256, 128
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3).cuda()
    layer, _ = layer_and_reference(E, H, I, x, idx, v, 9)
    x[2, 1] = float("nan")
    ctx, buf = Context(R, E, K, T, H), LLBuffer(R, E, K, T, H, T)
    for out in (layer.forward(ctx, x, idx, v), layer.forward_ll(buf, x, idx, v)):
        assert torch.isnan(out[2, 1]).all() and int(torch.isnan(out).any(-1).sum()) == 1
    ctx.check()
    buf.check()


def quantised_reference(layer, E, H, x, idx, v):
    """The layer of the FP8 forms: x and h through the codec, y rounded to bf16, all else in 64 bits."""
    from expert_util import rows64

    def codec(r):  # divided by a tensor: torch multiplies by the reciprocal of a number, which moves x's many ties
        b = r.reshape(r.shape[0], -1, 128)
        sc = b.abs().amax(-1) / torch.full_like(b[..., 0], 448.0)
        c = (b / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return rows64(c.view(torch.uint8).reshape(r.shape), sc)
    X = codec(x.view(-1, H).float())
    J, V = idx.view(-1, idx.shape[-1]), v.view(-1, idx.shape[-1]).double()
    I = layer.w2.shape[2]
    ref = torch.zeros_like(X)
    for e in range(E):
        t, k = torch.nonzero(J == e, as_tuple=True)
        y = X[t] @ weight64(layer.w13[e], layer.w13_scales[e]).t()
        h = codec((silu64(y[:, :I]) * y[:, I:]).float())
        ref.index_add_(0, t, V[t, k][:, None] * (h @ weight64(layer.w2[e], layer.w2_scales[e]).t()).to(torch.bfloat16).double())
    return ref.view(x.shape)


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I", [(4, 8, 2, 40, 128, 128), (2, 16, 4, 100, 512, 384)])
def test_fp8_forms_against_the_quantised_layer(R, E, K, T, H, I):
    """Both sides round x and h by the codec: what is left is bf16 (2^-9 / sqrt(3) = 1.1e-3 in the mean square, for y and
    for the output) and codes that round the other way (2^-4 each, one in 10^4 at most: 6e-4).  A scale off by 1 % is
    seen."""
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    layer, _ = layer_and_reference(E, H, I, x, idx, v, 10)
    ref = quantised_reference(layer, E, H, x, idx, v)
    ctx, buf = Context(R, E, K, T, H), LLBuffer(R, E, K, T, H, T)
    over, low = layer.forward(ctx, x, idx, v), layer.forward_ll(buf, x, idx, v)
    ctx.check()
    buf.check()
    assert far(over, ref) < 4e-3 and far(low, ref) < 4e-3, (far(over, ref), far(low, ref))
    assert far(1.01 * over.float(), ref) > 4e-3                   # the bound's own strength
