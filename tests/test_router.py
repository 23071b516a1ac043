"""route, balance_loss and router_backward against 64 bits.

Bounds, before any run.  A score: the exponent's argument l - m is rounded (|l - m| 2^-24 of the result), expf and the
division add 5 units of 2^-23, a row's sum at most 32 + 5 + 1: (span + 48) 2^-23 of itself, with span the row's largest
|l - m| (for sigmoid |l|).  Sums over a sequence: at most 400 terms one after another for the sizes here, all positive.
Gradients: the same share of the sum of the magnitudes of their terms, then half a step of the logits' type."""
import ctypes
import math

import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import Context, _lib, router
from expert_util import gen, randn

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def choice_ref(logits, K, bias=None, mask=None, groups=1, topk_groups=1):
    """The definition, token by token: keys in 32 bits, NaN the largest, ties to the lowest expert."""
    l = logits.float().cpu()
    key = l if bias is None else l + bias.cpu()
    out = torch.full((*key.shape[:-1], K), -1, dtype=torch.int64)
    flat, res = key.reshape(-1, key.shape[-1]).tolist(), out.view(-1, K)
    keep = [True] * len(flat) if mask is None else mask.cpu().reshape(-1).bool().tolist()
    big = lambda v: (1, 0.0) if v != v else (0, v)  # noqa: E731
    E = key.shape[-1]
    size = E // groups
    for t, row in enumerate(flat):
        if not keep[t]:
            continue
        allowed = range(E)
        if groups > 1:
            score = []
            for g in range(groups):
                two = sorted(row[g * size:(g + 1) * size], key=big, reverse=True)[:2]
                score.append(float(torch.tensor(two, dtype=F32).sum()))
            best = sorted(range(groups), key=lambda g: (tuple(-v for v in big(score[g])), g))[:topk_groups]
            allowed = [e for e in range(E) if e // size in best]
        order = sorted((e for e in allowed if row[e] != -INF), key=lambda e: (tuple(-v for v in big(row[e])), e))[:K]
        res[t, :len(order)] = torch.tensor(order, dtype=torch.int64)
    return out


def scores64(logits, scoring):
    v = logits.double()
    if scoring == "softmax":
        return torch.softmax(v, -1), None, (v - v.amax(-1, keepdim=True))
    return torch.sigmoid(v), torch.sigmoid(v) * torch.sigmoid(-v), v


def span_of(shifted):
    return torch.where(torch.isfinite(shifted), shifted.abs(), 0.0).amax(-1, keepdim=True)


def weights64(logits, idx, scoring, normalize):
    """(weights, by what a sigmoid was divided, the chosen experts' slopes)."""
    p, slope, _ = scores64(logits, scoring)
    on, at = idx >= 0, idx.clamp(min=0)
    w = torch.where(on, p.gather(-1, at), 0.0)
    by = torch.ones_like(w[..., :1])
    if normalize and scoring == "softmax":
        lv = torch.where(on, logits.double().gather(-1, at), -INF)
        w = torch.where(on, torch.softmax(lv, -1), 0.0)
    elif normalize:
        by = w.sum(-1, keepdim=True) + 1e-20
        w = w / by
    return w, by, None if slope is None else torch.where(on, slope.gather(-1, at), 0.0)


def assert_within(got, ref, lim, what=""):
    d = (got.double() - ref).abs()
    assert (d <= lim + 1e-37).all(), f"{what}: worst {float((d / (lim + 1e-37)).max()):.3g} of the bound"


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 33, 4), (40, 6, 6), (37, 64, 5), (33, 100, 8), (20, 128, 1), (64, 160, 6), (50, 256, 8), (9, 384, 32), (7, 512, 10),
          (5, 1000, 17), (3, 1024, 32)]


@gpu
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route(T, E, K, dtype, scoring, normalize):
    g = gen(T * E + K)
    logits = (2 * randn((T, E), g)).to(dtype)
    bias = 0.3 * randn((E,), g) if K % 2 == 0 else None
    mask = torch.rand(T, generator=g, device="cuda") < 0.8 if K % 2 == 0 else None
    idx, w = ep.route(logits, K, bias=bias, mask=mask, scoring=scoring, normalize=normalize, scale=2.5)
    assert torch.equal(idx.cpu(), choice_ref(logits, K, bias, mask))
    ref = 2.5 * weights64(logits, idx, scoring, normalize)[0]
    span = span_of(scores64(logits, scoring)[2])
    assert_within(w, ref, (span + 48) * 2.0 ** -23 * ref)


@gpu
@pytest.mark.parametrize("E,groups,topk_groups,K", [(8, 4, 2, 3), (64, 8, 4, 8), (256, 8, 4, 8), (256, 8, 1, 8), (96, 8, 3, 6), (160, 8, 3, 6), (100, 20, 7, 9),
                                                    (32, 32, 5, 5), (1024, 32, 2, 32), (12, 3, 3, 4), (6, 2, 1, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_by_groups(E, groups, topk_groups, K, dtype):
    g = gen(E + groups)
    logits = randn((41, E), g).to(dtype)
    logits[3] = 0                                               # all tied
    logits[4] = logits[4].round()                               # many ties
    logits[5, : E // 2] = -INF
    logits[6] = -INF
    logits[7, E - 1] = float("nan")
    logits[8, 0], logits[8, 1] = INF, -INF
    bias = 0.1 * randn((E,), g)
    for b in (None, bias):
        idx, _ = ep.route(logits, K, bias=b, scoring="sigmoid", groups=groups, topk_groups=topk_groups)
        assert torch.equal(idx.cpu(), choice_ref(logits, K, b, None, groups, topk_groups))


@gpu
def test_route_ties_infinities_nan_and_lowest_values():
    E, K = 40, 5
    low = torch.finfo(F32).min
    l = torch.zeros(9, E, device="cuda")
    l[1] = -INF                                                 # nothing to choose
    l[2] = -INF
    l[2, 30], l[2, 7] = 1.0, 2.0                                # two left of five
    l[3] = low                                                  # the type's lowest value is a value
    l[4] = low
    l[4, 39] = 1.0
    l[5, 11] = float("nan")
    l[6, 3] = -float("nan")
    l[7, ::2] = -0.0                                            # both zeros are equal
    l[8] = torch.arange(E, device="cuda").float()
    for scoring in ("softmax", "sigmoid"):
        idx, w = ep.route(l, K, scoring=scoring)
        assert torch.equal(idx.cpu(), choice_ref(l, K))
        assert idx[1].tolist() == [-1] * 5 and (w[1] == 0).all()
        assert idx[2].tolist() == [7, 30, -1, -1, -1] and (w[2, 2:] == 0).all()
        assert idx[3].tolist() == [0, 1, 2, 3, 4] and idx[4].tolist() == [39, 0, 1, 2, 3]
        assert idx[5, 0] == 11 and idx[6, 0] == 3 and torch.isnan(w[5]).all() and torch.isnan(w[6]).all()
        assert idx[7].tolist() == [0, 1, 2, 3, 4]
        ok = [0, 2, 4, 7, 8]
        assert ((w[ok].double().sum(-1) - 1).abs() < 1e-6).all()
    assert (ep.route(l, K)[1][3] - 0.2).abs().max() < 1e-7
    assert (ep.route(l, K, scoring="sigmoid")[1][3] == 0).all() # scores of 0 over 1e-20


@gpu
def test_route_strides_odd_rows_outputs_and_streams():
    g = gen(9)
    wide = randn((3, 7, 83), g)
    logits = wide[..., 2:79]                                    # 77 experts, rows 83 apart
    want = ep.route(logits.contiguous(), 6)
    idx = torch.full((3, 7, 6), 5, device="cuda", dtype=torch.int64)
    w = torch.full((3, 7, 6), 5.0, device="cuda")
    got = ep.route(logits, 6, out=(idx, w))
    assert got[0] is idx and torch.equal(idx, want[0]) and torch.equal(w, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ep.route(logits, 6, stream=side)
    side.synchronize()
    assert torch.equal(again[0], idx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = ep.route(logits, 6)
        bal = ep.balance_loss(logits, cap[0])
        dl = ep.router_backward(logits, cap[0], cap[1], factors=bal["factors"], dloss=torch.ones(1, device="cuda"))
    wide.copy_(randn((3, 7, 83), g))
    for _ in range(3):
        graph.replay()
    want = ep.route(logits, 6)
    b = ep.balance_loss(logits, want[0])
    assert torch.equal(cap[0], want[0]) and torch.equal(cap[1], want[1])
    assert torch.equal(bal["loss"], b["loss"]) and torch.equal(bal["counts"], b["counts"])
    assert torch.equal(dl, ep.router_backward(logits, want[0], want[1], factors=b["factors"], dloss=torch.ones(1, device="cuda")))


def balance64(logits, idx, coef, scoring):
    S, T, E = logits.shape
    p, _, shifted = scores64(logits, scoring)
    q = p if scoring == "softmax" else p / p.sum(-1, keepdim=True)
    used = (idx >= 0).any(-1)
    counts = torch.stack([torch.bincount(r[r >= 0], minlength=E) for r in idx.reshape(S, -1)])
    m, n = counts.sum(1).double().clamp(min=1), used.sum(1).double().clamp(min=1)
    F = coef * E * counts.double() / (S * m * n)[:, None]
    mass = (q * used[..., None]).sum(1)
    return (F * mass).sum(), counts, F, q, used, span_of(shifted)


BALANCE = [(1, 1, 4, 2), (4, 40, 8, 2), (3, 65, 33, 5), (2, 300, 100, 8), (5, 128, 256, 8), (1, 1000, 160, 6), (2, 50, 512, 16), (2, 9, 1024, 32), (70, 3, 16, 1)]


@gpu
@pytest.mark.parametrize("S,T,E,K", BALANCE)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_loss_and_its_gradient(S, T, E, K, dtype, scoring):
    g = gen(S * T + E)
    logits = (randn((S, T, E), g) + randn((E,), g)).to(dtype)
    mask = torch.rand((S, T), generator=g, device="cuda") < 0.85
    mask[0, 0] = True
    idx, _ = ep.route(logits, K, mask=mask)
    got = ep.balance_loss(logits, idx, 0.5, scoring=scoring)
    loss, counts, F, q, used, span = balance64(logits, idx, 0.5, scoring)
    assert torch.equal(got["counts"].long(), counts)
    assert_within(got["loss"][0], loss, (span.max() + 400) * 2.0 ** -23 * loss, "loss")
    centred = F - F.mean(-1, keepdim=True)
    assert_within(got["factors"], centred, 2.0 ** -22 * centred.abs(), "factors")
    dl = ep.router_backward(logits, idx, factors=got["factors"], dloss=torch.full((1,), 3.0, device="cuda"), scoring=scoring)
    f = centred[:, None]
    inner = (f * q).sum(-1, keepdim=True)
    mag_inner = (f.abs() * q).sum(-1, keepdim=True)
    if scoring == "softmax":
        ref, mag = 3 * q * (f - inner), 3 * q * (f.abs() + mag_inner)
    else:
        p, slope, _ = scores64(logits, scoring)
        by = 3 * slope / p.sum(-1, keepdim=True)
        ref, mag = by * (f - inner), by * (f.abs() + mag_inner)
    ref, mag = ref * used[..., None], mag * used[..., None]
    assert dl.dtype == dtype
    assert_within(dl, ref, HALF[dtype] * ref.abs() + 4 * (span + 96) * 2.0 ** -23 * mag, "dlogits")
    again = ep.balance_loss(logits, idx, 0.5, scoring=scoring)
    assert all(torch.equal(again[k], got[k]) for k in got)


@gpu
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("scoring,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_of_the_weights(T, E, K, scoring, normalize):
    g = gen(T + E)
    for dtype in (F32, BF):
        logits = randn((T, E), g).to(dtype)
        mask = torch.rand(T, generator=g, device="cuda") < 0.8
        idx, _ = ep.route(logits, K, mask=mask)
        dw = randn((T, K), g)
        got = ep.router_backward(logits, idx, dw, scoring=scoring, normalize=normalize, scale=1.5)
        w, by, slope = weights64(logits, idx, scoring, normalize)
        d = torch.where(idx >= 0, 1.5 * dw.double(), 0.0)
        inner, mag_inner = (d * w).sum(-1, keepdim=True), (d.abs() * w).sum(-1, keepdim=True)
        ref, mag = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda"), torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
        if scoring == "softmax":
            near, near_mag = (w * (d - inner), w * (d.abs() + mag_inner)) if normalize else (w * d, w * d.abs())
        else:
            near, near_mag = (slope / by * (d - inner), slope / by * (d.abs() + mag_inner)) if normalize else (slope * d, slope * d.abs())
        at = torch.where(idx >= 0, idx, E)
        ref, mag = ref.scatter_add(1, at, near)[:, :E], mag.scatter_add(1, at, near_mag)[:, :E]
        if scoring == "softmax" and not normalize:
            p = scores64(logits, scoring)[0] * mask[:, None]
            ref, mag = ref - p * inner, mag + p * mag_inner
        span = span_of(scores64(logits, scoring)[2])
        assert_within(got, ref, HALF[dtype] * ref.abs() + 4 * (span + 96) * 2.0 ** -23 * mag)
        if not bool(mask.all()):
            assert (got[~mask] == 0).all()


@gpu
@pytest.mark.parametrize("scoring,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradients_against_differences(scoring, normalize):
    """Weights and loss together along a direction, against the 64-bit forward's central difference."""
    S, T, E, K = 2, 6, 20, 4
    g = gen(5)
    logits = randn((S, T, E), g)
    idx, _ = ep.route(logits, K)
    dw = randn((S, T, K), g)
    bal = ep.balance_loss(logits, idx, 0.7, scoring=scoring)
    got = ep.router_backward(logits, idx, dw, factors=bal["factors"], dloss=torch.full((1,), 2.0, device="cuda"), scoring=scoring,
                             normalize=normalize)
    u, t = randn((S, T, E), g).double(), 1e-4

    def f(k):
        l = logits.double() + k * u
        return (dw.double() * weights64(l, idx, scoring, normalize)[0]).sum() + 2 * balance64(l, idx, 0.7, scoring)[0]
    numeric = (f(t) - f(-t)) / (2 * t)
    exact = (got.double() * u).sum()
    assert abs(numeric - exact) <= 1e-4 * (got.double() * u).abs().sum()


@gpu
def test_same_expert_twice_padding_and_empty_sequences():
    E, K = 12, 3
    g = gen(6)
    logits = randn((3, 4, E), g)
    idx = torch.full((3, 4, K), -1, device="cuda", dtype=torch.int64)
    idx[0, 1] = torch.tensor([5, 5, 2])
    idx[2, :, 0] = 7                                            # sequence 1 is empty
    got = ep.balance_loss(logits, idx)
    loss, counts, F, q, used, span = balance64(logits, idx, 1.0, "softmax")
    assert torch.equal(got["counts"].long(), counts) and counts[0, 5] == 2 and (counts[1] == 0).all()
    assert (got["factors"][1] == 0).all()
    assert_within(got["loss"][0], loss, 500 * 2.0 ** -23 * loss)
    dw = torch.zeros(3, 4, K, device="cuda")
    dw[0, 1] = torch.tensor([1.0, 2.0, 4.0])
    dl = ep.router_backward(logits, idx, dw)
    l = logits[0, 1].double().requires_grad_()
    w = torch.softmax(l[idx[0, 1]], 0)
    (w * dw[0, 1].double()).sum().backward()
    assert (dl[0, 1].double() - l.grad).abs().max() < 1e-6
    dl[0, 1] = 0
    assert (dl == 0).all()


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_padding_may_hold_anything_and_closed_experts_get_nothing(scoring):
    S, T, E, K = 3, 50, 40, 4
    logits = randn((S, T, E), gen(21))
    logits[..., [3, 17, 39]] = -INF                             # closed
    logits[..., 5] = torch.finfo(F32).min
    mask = torch.rand((S, T), generator=gen(22), device="cuda") < 0.7
    clean = ep.route(logits, K, mask=mask, scoring=scoring)
    dw = randn((S, T, K), gen(23))
    one = torch.ones(1, device="cuda")

    def step(l, d):
        idx, w = ep.route(l, K, mask=mask, scoring=scoring)
        bal = ep.balance_loss(l, idx, scoring=scoring)
        return idx, w, bal["loss"], bal["counts"], ep.router_backward(l, idx, d, factors=bal["factors"], dloss=one, scoring=scoring)
    want = step(logits, dw)
    assert torch.equal(want[0], clean[0]) and not torch.isin(want[0], torch.tensor([3, 17, 39], device="cuda")).any()
    assert torch.isfinite(want[2]).all() and torch.isfinite(want[4]).all()
    assert (want[4][..., [3, 17, 39]] == 0).all() and (want[4][~mask] == 0).all() and (want[3][:, [3, 17, 39]] == 0).all()
    dirty, d = logits.clone(), dw.clone()
    dirty[~mask] = float("nan")
    dirty[0, ~mask[0]] = INF
    d[~mask] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(step(dirty, d), want))


@gpu
def test_given_outputs_and_workspaces():
    l = randn((3, 40, 24), gen(24))
    idx, _ = ep.route(l, 2)
    want = ep.balance_loss(l, idx, 0.3)
    out = {k: torch.full_like(v, 9) for k, v in want.items()}
    ws = torch.full((ep.balance_loss_workspace(120, 24, 3),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = ep.balance_loss(l, idx, 0.3, out=out, workspace=ws)
        assert all(got[k] is out[k] and torch.equal(got[k], want[k]) for k in want)
    with pytest.raises(ep.EpError):
        ep.balance_loss(l, idx, workspace=ws[:-16])
    with pytest.raises(ValueError):
        ep.balance_loss(l, idx, out=out | {"counts": out["loss"]})


@gpu
def test_entries_out_of_range_are_skipped_and_reported():
    logits = randn((6, 8), gen(7))
    idx = torch.zeros(6, 2, device="cuda", dtype=torch.int64)
    idx[:, 1] = 3
    bad = idx.clone()
    bad[2, 0], bad[3, 1], bad[4, 0] = 8, -2, 1 << 40
    idx[2, 0] = idx[3, 1] = idx[4, 0] = -1
    status = ep.new_status()
    want, got = ep.balance_loss(logits, idx, status=status), None
    ep.check_status(status)
    got = ep.balance_loss(logits, bad, status=status)
    assert all(torch.equal(got[k], want[k]) for k in want)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(status)
    assert e.value.code == -2
    dw = torch.ones(6, 2, device="cuda")
    assert torch.equal(ep.router_backward(logits, bad, dw, normalize=False, status=status), ep.router_backward(logits, idx, dw, normalize=False))
    with pytest.raises(ep.EpError):
        ep.check_status(status)


@gpu
def test_rows_further_apart_than_32_bits_reach():
    E, far = 72, (1 << 30) + 8
    big = torch.empty(3 * far, dtype=BF, device="cuda")
    l = torch.as_strided(big, (3, E), (far, 1))
    l.copy_(randn((3, E), gen(12)))
    c = l.clone()
    idx, w = ep.route(l, 5)
    want = ep.route(c, 5)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    got, ref = ep.balance_loss(l, idx), ep.balance_loss(c, idx)
    assert all(torch.equal(got[k], ref[k]) for k in ref)
    one = torch.ones(1, device="cuda")
    want = ep.router_backward(c, idx, w, factors=ref["factors"], dloss=one)
    assert torch.equal(ep.router_backward(l, idx, w, factors=ref["factors"], dloss=one, out=l), want)


@gpu
@pytest.mark.parametrize("S,T,E,K", [(1, 20011, 256, 8), (3, 9001, 33, 4), (2, 7001, 160, 6), (5, 3333, 512, 10), (1, 9999, 1000, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_tokens_than_one_wave(S, T, E, K, dtype):
    """Every warp has several tokens, some of them padded; the choice against a stable sort, all else as above."""
    g = gen(S * T)
    logits = (randn((S, T, E), g) + randn((E,), g)).to(dtype)
    mask = torch.rand((S, T), generator=g, device="cuda") < 0.9
    idx, w = ep.route(logits, K, mask=mask)
    want = torch.sort(logits.float(), dim=-1, descending=True, stable=True).indices[..., :K]
    assert torch.equal(idx, torch.where(mask[..., None], want, -1))
    span = span_of(scores64(logits, "softmax")[2])
    ref = weights64(logits, idx, "softmax", True)[0]
    assert_within(w, ref, (span + 48) * 2.0 ** -23 * ref)
    got = ep.balance_loss(logits, idx)
    loss, counts, F, q, used, _ = balance64(logits, idx, 1.0, "softmax")
    assert torch.equal(got["counts"].long(), counts)
    # a warp adds at most T / 600 tokens of a sequence (or 2 * 8 a block), then 8 warps, at most 608 blocks
    assert_within(got["loss"][0], loss, (span.max() + T / 600 + 700) * 2.0 ** -23 * loss, "loss")
    dw = randn((S, T, K), g)
    one = torch.ones(1, device="cuda")
    dl = ep.router_backward(logits, idx, dw, factors=got["factors"], dloss=one)
    f = (F - F.mean(-1, keepdim=True))[:, None]
    inner, mag_inner = (f * q).sum(-1, keepdim=True), (f.abs() * q).sum(-1, keepdim=True)
    d = torch.where(idx >= 0, dw.double(), 0.0)
    near = ref * (d - (d * ref).sum(-1, keepdim=True))
    near_mag = ref * (d.abs() + (d.abs() * ref).sum(-1, keepdim=True))
    at = idx.clamp(min=0)
    want = (q * (f - inner) * used[..., None]).scatter_add(-1, at, near)
    mag = (q * (f.abs() + mag_inner)).scatter_add(-1, at, near_mag)
    assert_within(dl, want, HALF[dtype] * want.abs() + 4 * (span + 96) * 2.0 ** -23 * mag, "dlogits")
    same = ep.router_backward(logits, idx, dw, factors=got["factors"], dloss=one, out=logits)
    assert same is logits and torch.equal(same, dl)


@gpu
def test_no_tokens_and_in_place_gradient():
    l = torch.empty(0, 16, device="cuda")
    idx, w = ep.route(l, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    got = ep.balance_loss(l, idx)
    assert got["loss"].item() == 0 and (got["counts"] == 0).all() and (got["factors"] == 0).all()
    assert ep.router_backward(l, idx, w).shape == (0, 16)
    l = randn((9, 37), gen(1))
    idx, w = ep.route(l, 4)
    want = ep.router_backward(l, idx, w)
    got = ep.router_backward(l, idx, w, out=l)
    assert got is l and torch.equal(got, want)


@gpu
def test_a_contexts_routes_reach_no_more_nodes_than_asked():
    R, E, K, T, N = 8, 64, 6, 30, 4
    ctx = Context(R, E, K, T, 128, num_nodes=N)
    logits = randn((R, T, E), gen(2))
    idx, w = ctx.route(logits, topk_nodes=2, scoring="sigmoid")
    assert torch.equal(idx.cpu(), choice_ref(logits, K, None, None, N, 2))
    lay = ctx.get_dispatch_layout(idx)
    ctx.check()
    assert int(lay["is_token_in_node"].sum(-1).max()) <= 2
    assert torch.equal(lay["num_tokens_per_expert"], ep.balance_loss(logits, idx)["counts"])
    with pytest.raises(ValueError):
        ctx.route(logits[:2])


def test_refusals_of_the_binding():
    l = torch.zeros(4, 8)
    for call in (lambda: ep.route(l, 2), lambda: ep.balance_loss(l, l), lambda: ep.router_backward(l, l)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@gpu
def test_refusals_on_the_gpu():
    l = torch.zeros(4, 8, device="cuda")
    idx, w = ep.route(l, 2)
    one = torch.ones(1, device="cuda")
    f = torch.zeros(1, 8, device="cuda")
    for call in (lambda: ep.route(l.half(), 2), lambda: ep.route(l, 2, scoring="relu"), lambda: ep.route(l, 2, bias=l[0, :4]),
                 lambda: ep.route(l, 2, mask=torch.ones(3, device="cuda", dtype=torch.bool)), lambda: ep.route(l[:, ::2], 2),
                 lambda: ep.route(l, 2, out=(idx.int(), w)), lambda: ep.balance_loss(l, idx.int()), lambda: ep.balance_loss(l, idx[:2]),
                 lambda: ep.router_backward(l, idx, w.double()), lambda: ep.router_backward(l, idx, factors=f[:, :4], dloss=one),
                 lambda: ep.router_backward(l, idx, w, out=l.to(BF))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ep.route(l, 9), lambda: ep.route(l, 0), lambda: ep.route(l, 2, groups=3), lambda: ep.route(l, 3, groups=4, topk_groups=1),
                 lambda: ep.router_backward(l, idx), lambda: ep.router_backward(l, idx, factors=f),
                 lambda: ep.balance_loss(l, idx, workspace=torch.empty(16, device="cuda", dtype=torch.uint8)),
                 lambda: ep.route(torch.zeros(1, 1025, device="cuda"), 2)):
        with pytest.raises(ep.EpError):
            call()


GOOD = dict(tokens=4, experts=8, topk=2, logits_type=1, scoring=0, normalize=1, groups=1, topk_groups=1, scale=1.0)


@pytest.mark.parametrize("change", [dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=9), dict(topk=33, experts=64),
                                    dict(logits_type=2), dict(scoring=-1), dict(groups=0), dict(groups=3), dict(groups=33, experts=66),
                                    dict(topk_groups=2), dict(topk_groups=0), dict(groups=8, topk_groups=1)])
def test_refusals_of_the_library(change):
    """Addresses that are never read: every call is refused on the host."""
    a = GOOD | change
    r = router._ROUTER(a["tokens"], a["experts"], a["topk"], a["logits_type"], a["scoring"], a["normalize"], a["groups"], a["topk_groups"], a["scale"])
    assert len(r) == ctypes.sizeof(_lib.EpRouter)
    assert _lib.load().ep_route(r, 0x1000, a["experts"], None, None, 0x2000, 0x3000, None) == -1
    assert _lib.load().ep_last_error().startswith(b"ep_route:")


@pytest.mark.parametrize("call", [
    lambda lib, r: lib.ep_route(None, 0x1000, 8, None, None, 0x2000, 0x3000, None),
    lambda lib, r: lib.ep_route(r, None, 8, None, None, 0x2000, 0x3000, None),
    lambda lib, r: lib.ep_route(r, 0x1002, 8, None, None, 0x2000, 0x3000, None),
    lambda lib, r: lib.ep_route(r, 0x1000, 7, None, None, 0x2000, 0x3000, None),
    lambda lib, r: lib.ep_route(r, 0x1000, 8, 0x1001, None, 0x2000, 0x3000, None),
    lambda lib, r: lib.ep_route(r, 0x1000, 8, None, None, 0x2004, 0x3000, None),
    lambda lib, r: lib.ep_route(r, 0x1000, 8, None, None, 0x2000, None, None),
    lambda lib, r: lib.ep_balance_loss(r, 0x1000, 8, 0x2000, 3, 1.0, 0x3000, 0x4000, 0x5000, 0x6000, 1 << 20, None, None),
    lambda lib, r: lib.ep_balance_loss(r, 0x1000, 8, None, 1, 1.0, 0x3000, 0x4000, 0x5000, 0x6000, 1 << 20, None, None),
    lambda lib, r: lib.ep_balance_loss(r, 0x1000, 8, 0x2000, 1, 1.0, None, 0x4000, 0x5000, 0x6000, 1 << 20, None, None),
    lambda lib, r: lib.ep_balance_loss(r, 0x1000, 8, 0x2000, 1, 1.0, 0x3000, 0x4001, 0x5000, 0x6000, 1 << 20, None, None),
    lambda lib, r: lib.ep_router_backward(r, 0x1000, 8, 0x2000, None, None, 1, None, 0x7000, 8, None, None),
    lambda lib, r: lib.ep_router_backward(r, 0x1000, 8, 0x2000, 0x3000, 0x4000, 1, None, 0x7000, 8, None, None),
    lambda lib, r: lib.ep_router_backward(r, 0x1000, 8, 0x2000, 0x3000, 0x4000, 3, 0x5000, 0x7000, 8, None, None),
    lambda lib, r: lib.ep_router_backward(r, 0x1000, 8, 0x2000, 0x3000, None, 1, None, 0x7000, 4, None, None),
    lambda lib, r: lib.ep_router_backward(r, 0x1000, 8, 0x2000, 0x3000, None, 1, None, None, 8, None, None),
])
def test_refused_calls_of_the_library(call):
    r = router._ROUTER(*GOOD.values())
    assert call(_lib.load(), r) == -1
