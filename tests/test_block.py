"""Norm, router, balance loss and experts together, as a mixture-of-experts block uses them: a serving step with 8- and 4-bit
experts, and a training step's gradients through the norm and the router."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import Context, inputs
from combine_get_dispatch_histograms_gb300.layer import MoELayer
from expert_util import gen, quantize_weight, randn, silu64, weight64
from test_fp4 import quantize_ref, values4, weight4

gpu = pytest.mark.gpu
BF = torch.bfloat16


def experts64(X, J, V, w13, w2, codec=None):
    """sum_k V W2 (silu(Wg x) * (Wu x)) in 64 bits; codec: what h passes through, with y in bf16."""
    out = torch.zeros_like(X)
    for e in range(w13.shape[0]):
        t, k = torch.nonzero(J == e, as_tuple=True)
        y = X[t] @ w13[e].t()
        n = y.shape[1] // 2
        h = silu64(y[:, :n]) * y[:, n:]
        y = h @ w2[e].t() if codec is None else (codec(h) @ w2[e].t()).to(BF).double()
        out.index_add_(0, t, V[t, k][:, None] * y)
    return out


def block(R, E, K, T, H, seed):
    g = gen(seed)
    x = inputs.random_x(R, T, H, seed).cuda()
    r = (2 * randn((R, T, H), g)).to(BF)
    return g, x, r, 1 + 0.1 * randn((H,), g), randn((E, H), g) * H ** -0.5


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I", [(4, 8, 2, 40, 256, 128), (2, 16, 4, 100, 512, 384)])
@pytest.mark.parametrize("fp4", [False, True])
def test_a_serving_step(R, E, K, T, H, I, fp4):
    g, x, r, wn, wr = block(R, E, K, T, H, 5)
    w13, w2 = randn((E, 2 * I, H), g) * H ** -0.5, randn((E, H, I), g) * I ** -0.5
    if fp4:
        (w13, s13), (w2, s2) = weight4(E, 2 * I, H, g), weight4(E, H, I, g)
        m13, m2 = (torch.stack([values4(w[e], s[e]) for e in range(E)]) for w, s in ((w13, s13), (w2, s2)))
    else:
        (w13, s13), (w2, s2) = quantize_weight(w13), quantize_weight(w2)
        m13, m2 = (torch.stack([weight64(w[e], s[e]) for e in range(E)]) for w, s in ((w13, s13), (w2, s2)))
    ctx, layer = Context(R, E, K, T, H), MoELayer(w13, s13, w2, s2)

    def step():
        got = ep.rms_norm(x, wn, residual=r)
        idx, w = ctx.route(got["y"].float() @ wr.t())
        return got["residual"], got["y"], idx, w, layer.forward(ctx, got["y"], idx, w)
    h, y, idx, w, out = step()
    ctx.check()
    total = (x.double() + r.double()).float().to(BF)
    assert torch.equal(h, total)
    codec = None
    X = y.view(-1, H).double()
    if fp4:  # both sides round x and h by the codec: what is left is bf16, and codes that round the other way (see test_fp4)
        codec = lambda v: values4(*quantize_ref(v))  # noqa: E731
        X = codec(X)
    ref = experts64(X, idx.view(-1, K), w.view(-1, K).double(), m13, m2, codec)
    assert float((out.view(-1, H).double() - ref).norm() / ref.norm()) < (5e-3 if fp4 else 0.12)
    # the same captured, on new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    x.copy_(inputs.random_x(R, T, H, 77).cuda())
    graph.replay()
    ctx.check()
    assert all(torch.equal(a, b) for a, b in zip(cap, step()))


@gpu
@pytest.mark.parametrize("scoring,normalize", [("softmax", True), ("sigmoid", True), ("softmax", False)])
def test_a_training_steps_gradients(scoring, normalize):
    """x and r through norm and router to weights and loss, against 64-bit autograd from the same choice.  The rounding of y
    to bf16 is 2^-8 of it at most, so the gradients agree to a few 2^-8 of their norm: held to 2^-5."""
    R, E, K, T, H = 2, 16, 4, 50, 256
    g, x, r, wn, wr = block(R, E, K, T, H, 9)
    r = r.float()
    got = ep.rms_norm(x, wn, residual=r)
    y, h = got["y"], got["residual"]
    logits = y.float() @ wr.t()
    idx, w = ep.route(logits, K, scoring=scoring, normalize=normalize)
    bal = ep.balance_loss(logits, idx, coef=3.0, scoring=scoring)
    dw = randn((R, T, K), g)
    dl = ep.router_backward(logits, idx, dw, factors=bal["factors"], dloss=torch.ones(1, device="cuda"), scoring=scoring, normalize=normalize)
    dy = (dl @ wr).to(BF)
    dx, dwn = ep.rms_norm_backward(dy, h, wn)

    h64, n64 = h.double().requires_grad_(), wn.double().requires_grad_()
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * n64
    l64 = y64 @ wr.double().t()
    p = torch.softmax(l64, -1) if scoring == "softmax" else torch.sigmoid(l64)
    q = p if scoring == "softmax" else p / p.sum(-1, keepdim=True)
    picked = p.gather(-1, idx)
    if normalize:
        picked = picked / picked.sum(-1, keepdim=True)
    counts = torch.stack([torch.bincount(i.view(-1), minlength=E) for i in idx]).double()
    loss = 3.0 * (E * counts / counts.sum(1, keepdim=True) * q.mean(1)).sum() / R
    ((picked * dw.double()).sum() + loss).backward()
    assert abs(float(bal["loss"]) - float(loss.detach())) < 2.0 ** -7 * float(loss.detach())
    for a, b in ((dx, h64.grad), (dwn, n64.grad)):
        assert float((a.double() - b).norm() / b.norm()) < 2.0 ** -5


@gpu
def test_steps_that_share_buffers_without_waits():
    """Launches overlap: a step rewrites what the step before has just read, and reads what its own last kernel wrote."""
    S, T, E, K, H, I = 2, 200, 64, 4, 512, 256
    g = gen(31)
    steps = range(9)
    xs = [randn((S * T, H), g).to(BF) * 2.0 ** (i - 4) for i in steps]  # scales differ from step to step
    wn, wr = 1 + 0.1 * randn((H,), g), randn((E, H), g) * H ** -0.5
    logits = [(x.float() @ wr.t()).view(S, T, E) for x in xs]
    (w13, s13), (w2, s2) = weight4(1, 2 * I, H, g), weight4(1, H, I, g)
    dw, one = randn((S, T, K), g), torch.ones(1, device="cuda")
    empty = lambda *s, t=torch.uint8: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    F32 = torch.float32

    def buffers():
        return dict(norm=dict(y=empty(S * T, H, t=BF)), route=(empty(S, T, K, t=torch.int64), empty(S, T, K, t=F32)),
                    balance=dict(loss=empty(1, t=F32), counts=empty(S, E, t=torch.int32), factors=empty(S, E, t=F32)),
                    workspace=empty(ep.balance_loss_workspace(S * T, E, S)), q=(empty(S * T, H // 2), empty(S * T, H // 32)),
                    h=(empty(S * T, I // 2), empty(S * T, I // 32)))

    def step(i, b, out):
        idx, _ = ep.route(logits[i], K, out=b["route"])
        factors = ep.balance_loss(logits[i], idx, out=b["balance"], workspace=b["workspace"])["factors"]
        ep.router_backward(logits[i], idx, dw, factors=factors, dloss=one, out=out[0])
        y = ep.rms_norm(xs[i], wn, out=b["norm"])["y"]
        ep.quantize_fp4(xs[i] if i % 2 else y, out=b["q"])
        ep.expert_swiglu_fp4(*b["q"], w13, s13, out=b["h"])
        ep.expert_gemm_fp4(*b["h"], w2, s2, out=out[1])
    outs = lambda: [(empty(S, T, E, t=F32), empty(S * T, H, t=BF)) for _ in steps]  # noqa: E731
    alone, got, shared = outs(), outs(), buffers()
    for i in steps:
        step(i, buffers(), alone[i])
        torch.cuda.synchronize()
    assert len({float(y.float().norm()) for _, y in alone}) == len(steps)

    def run():
        for i in steps:
            step(i, shared, got[i])
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for _ in range(20):
        for o in got:
            for t in o:
                t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for x, y in zip(alone, got) for a, b in zip(x, y))


def test_layer_refuses_mixed_weights():
    u8, f32 = torch.zeros(1, dtype=torch.uint8), torch.zeros(1)
    with pytest.raises(ValueError):
        MoELayer(u8, u8, u8, f32)
    with pytest.raises(ValueError):
        MoELayer(u8, u8, u8, u8).forward_ll(None, None, None, None)
