"""route by keys made of scores, against the definition in 64 bits, token by token.

Bounds, before any run.  A score is off by at most (span + 48) 2^-23 of itself (test_router), a key by half a step of the sum
more, a group's sum by its two keys' and half a step.  Two keys nearer than that may come in either order: such tokens are left
out, and are few, unless both have the same logit and bias: then the lower expert comes first."""
import math

import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import Context, _lib, router
from expert_util import gen, randn
from test_router import BF, F32, GOOD, INF, assert_within, scores64, span_of, weights64

gpu = pytest.mark.gpu


def choose64(logits, bias, scoring, K, groups=1, topk_groups=1, group_keys=2):
    """Per token the experts in order, or None where rounding may decide."""
    l = logits.double().cpu()
    E = l.shape[-1]
    score, _, shifted = scores64(l, scoring)
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    key = torch.where(l == -INF, -INF, score + b)
    eps = torch.where(l == -INF, 0.0, (span_of(shifted) + 48) * 2.0 ** -23 * score + 2.0 ** -24 * key.abs())
    out = []
    for row, err, at in zip(key.tolist(), eps.tolist(), l.tolist()):
        size, allowed, clear = E // groups, list(range(E)), True
        if topk_groups < groups:
            counted = []
            for g in range(groups):
                two = sorted(range(g * size, g * size + size), key=lambda e: -row[e])[:min(group_keys, size)]
                v = sum(row[e] for e in two)
                counted.append((v, sum(err[e] for e in two) + (2.0 ** -24 * abs(v) if math.isfinite(v) else 0)))
            best = sorted(range(groups), key=lambda g: (-counted[g][0], g))
            (a, ea), (c, ec) = counted[best[topk_groups - 1]], counted[best[topk_groups]]
            clear = a == c == -INF or a - c > ea + ec
            allowed = [e for e in allowed if e // size in best[:topk_groups]]
        order = sorted((e for e in allowed if row[e] != -INF), key=lambda e: (-row[e], e))
        for i, j in zip(order[:K], order[1:K + 1]):
            clear &= row[i] - row[j] > err[i] + err[j] or (at[i], float(b[i])) == (at[j], float(b[j]))
        out.append(order[:K] + [-1] * (K - len(order[:K])) if clear else None)
    return out


def assert_chosen(idx, want, least):
    rows = idx.reshape(-1, idx.shape[-1]).tolist()
    clear = [i for i, w in enumerate(want) if w is not None]
    assert len(clear) >= least * len(want)
    assert [rows[i] for i in clear] == [want[i] for i in clear]


def test_the_definition_on_small_numbers():
    l = torch.tensor([[4.0, 3.0, 0.0, -1.0]])                   # sigmoids 0.982, 0.953, 0.5, 0.269
    assert choose64(l, torch.tensor([0.0, 0.0, 0.5, 0.0]), "sigmoid", 2) == [[2, 0]]
    l = torch.tensor([[8.0, -1.0, 3.0, 2.0]])                   # sums of logits 7 and 5, of sigmoids 1.27 and 1.83
    assert choose64(l, None, "sigmoid", 2, 2, 1) == [[2, 3]]
    assert choose64(l, None, "sigmoid", 2, 2, 1, group_keys=1) == [[0, 1]]


@gpu
def test_keys_of_scores_are_not_keys_of_logits():
    l, bias = torch.tensor([[4.0, 3.0, 0.0, -1.0]], device="cuda"), torch.tensor([0.0, 0.0, 0.5, 0.0], device="cuda")
    assert ep.route(l, 2, bias=bias, scoring="sigmoid", keys="scores")[0].tolist() == [[2, 0]]
    assert ep.route(l, 2, bias=bias, scoring="sigmoid")[0].tolist() == [[0, 1]]
    l = torch.tensor([[8.0, -1.0, 3.0, 2.0]], device="cuda")
    by = dict(scoring="sigmoid", groups=2, topk_groups=1)
    assert ep.route(l, 2, keys="scores", **by)[0].tolist() == [[2, 3]]
    assert ep.route(l, 2, **by)[0].tolist() == [[0, 1]]
    assert ep.route(l, 2, keys="scores", group_keys=1, **by)[0].tolist() == [[0, 1]]
    l = torch.tensor([[3.0, 3.0, 4.0, -9.0]], device="cuda")
    assert ep.route(l, 2, **by)[0].tolist() == [[0, 1]] and ep.route(l, 2, group_keys=1, **by)[0].tolist() == [[2, 3]]


@gpu
@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (33, 4), (64, 6), (100, 8), (256, 8), (384, 8), (1024, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_with_a_bias_on_the_scores(E, K, dtype, scoring, normalize):
    g = gen(E + K)
    T = 61
    logits = (1.5 * randn((T, E), g)).to(dtype)
    bias = (0.2 if scoring == "sigmoid" else 0.5 / E) * randn((E,), g)
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    idx, w = ep.route(logits, K, bias=bias, mask=mask, scoring=scoring, normalize=normalize, scale=2.5, keys="scores")
    want = choose64(logits, bias, scoring, K)
    want = [v if m else [-1] * K for v, m in zip(want, mask.tolist())]
    assert_chosen(idx, want, 0.7)
    ref = 2.5 * weights64(logits, idx, scoring, normalize)[0]   # of the scores alone
    assert_within(w, ref, (span_of(scores64(logits, scoring)[2]) + 48) * 2.0 ** -23 * ref)
    plain = ep.route(logits, K, scoring=scoring, keys="scores")[0]
    assert_chosen(plain, choose64(logits, None, scoring, K), 0.7)


@gpu
@pytest.mark.parametrize("E,groups,topk_groups,K", [(8, 4, 2, 3), (64, 8, 4, 8), (256, 8, 4, 8), (256, 8, 1, 8), (160, 8, 3, 6), (100, 20, 7, 9), (32, 32, 5, 5),
                                                    (1024, 32, 2, 32), (12, 3, 3, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_keys", [1, 2])
def test_route_by_groups_of_scores(E, groups, topk_groups, K, dtype, scoring, group_keys):
    g = gen(E + groups + group_keys)
    logits = randn((53, E), g).to(dtype)
    logits[3] = 0                                               # all tied
    logits[5, : E // 2] = -INF                                  # closed experts
    logits[6] = -INF
    bias = (0.1 if scoring == "sigmoid" else 0.2 / E) * randn((E,), g)
    for b in (None, bias):
        idx, _ = ep.route(logits, K, bias=b, scoring=scoring, groups=groups, topk_groups=topk_groups, keys="scores", group_keys=group_keys)
        assert_chosen(idx, choose64(logits, b, scoring, K, groups, topk_groups, group_keys), 0.6)
        assert (idx[6] == -1).all()
    first = ep.route(logits[3:4], K, scoring=scoring, groups=groups, topk_groups=topk_groups, keys="scores", group_keys=group_keys)[0]
    assert first.tolist() == [list(range(K))]                   # equal groups and keys: the lowest


@gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties_infinities_and_nan(scoring):
    E, K = 40, 5
    l = torch.zeros(8, E, device="cuda")
    l[1] = -INF
    l[2] = -INF
    l[2, 30], l[2, 7] = 1.0, 2.0                                # two left of five
    l[3] = torch.finfo(F32).min                                 # a value: softmaxes alike, sigmoids all 0
    l[4, 11] = float("nan")
    l[5, ::2] = -0.0
    l[6] = 30 + torch.arange(E, device="cuda")                  # sigmoids all 1
    l[7, 9] = INF
    idx, w = ep.route(l, K, scoring=scoring, keys="scores")
    low = [0, 1, 2, 3, 4]
    assert idx[0].tolist() == low and idx[1].tolist() == [-1] * K and idx[2].tolist() == [7, 30, -1, -1, -1] and idx[3].tolist() == low
    assert idx[4].tolist() == (low if scoring == "softmax" else [11, 0, 1, 2, 3])  # a softmax is NaN as a whole
    assert idx[5].tolist() == low and (w[1] == 0).all() and (w[2, 2:] == 0).all()
    assert idx[6].tolist() == (low if scoring == "sigmoid" else [39, 38, 37, 36, 35])
    assert idx[7].tolist() == (low if scoring == "softmax" else [9, 0, 1, 2, 3])
    bias = torch.zeros(E, device="cuda")
    bias[:3] = -INF                                             # closed by the bias, whatever the score
    assert ep.route(l[:1], K, bias=bias, scoring=scoring, keys="scores")[0].tolist() == [[3, 4, 5, 6, 7]]
    bias[0] = INF
    assert ep.route(l[1:3], K, bias=bias, scoring=scoring, keys="scores")[0].tolist() == [[-1] * K, [7, 30, -1, -1, -1]]


@gpu
def test_more_tokens_than_one_wave_strides_and_a_graph():
    """8 of 256 experts out of 4 of 8 groups, biased scores, by torch's own 32-bit sigmoid: as before, near ties left out."""
    T, E, K, G = 9001, 256, 8, 8
    g = gen(4)
    wide = randn((T, E + 8), g)
    logits, bias = wide[:, 3:E + 3], 0.2 * randn((E,), g)
    how = dict(bias=bias, scoring="sigmoid", groups=G, topk_groups=4, keys="scores", scale=2.5)
    graph = torch.cuda.CUDAGraph()
    want = ep.route(logits.contiguous(), K, **how)
    with torch.cuda.graph(graph):
        idx, w = ep.route(logits, K, **how)
    graph.replay()
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    key = torch.sigmoid(logits.double()) + bias
    two = key.view(T, G, -1).topk(2, -1).values.sum(-1)
    order = two.sort(-1, descending=True)
    keep = torch.zeros_like(two).scatter_(1, order.indices[:, :4], 1.0).bool().repeat_interleave(E // G, 1)
    top = key.masked_fill(~keep, -INF).sort(-1, descending=True)
    gap = (top.values[:, :K] - top.values[:, 1:K + 1]).amin(1)
    clear = (order.values[:, 3] - order.values[:, 4] > 1e-4) & (gap > 1e-4)  # keys below 2, |logits| below 6: errors below 54 2^-23 + 2^-23
    assert clear.float().mean() > 0.9
    assert torch.equal(idx[clear], top.indices[clear][:, :K])


@gpu
def test_a_contexts_route_by_scores():
    R, E, K, T, N = 8, 64, 6, 30, 4
    ctx = Context(R, E, K, T, 128, num_nodes=N)
    g = gen(2)
    logits, bias = randn((R, T, E), g), 0.3 * randn((E,), g)
    idx, w = ctx.route(logits, topk_nodes=2, scoring="sigmoid", bias=bias, keys="scores")
    assert_chosen(idx, choose64(logits.view(-1, E), bias, "sigmoid", K, N, 2), 0.9)
    lay = ctx.get_dispatch_layout(idx)
    ctx.check()
    assert int(lay["is_token_in_node"].sum(-1).max()) <= 2


@gpu
def test_refusals_on_the_gpu():
    l = torch.zeros(4, 8, device="cuda")
    for how in (dict(keys="bias"), dict(keys=None), dict(group_keys=0), dict(group_keys=3)):
        with pytest.raises(ValueError):
            ep.route(l, 2, **how)


@pytest.mark.parametrize("change", [dict(keys=-1), dict(keys=2), dict(group_keys=-1), dict(group_keys=3)])
def test_refusals_of_the_library(change):
    r = router._ROUTER(*GOOD.values(), **change)
    assert _lib.load().ep_route(r, 0x1000, 8, None, None, 0x2000, 0x3000, None) == -1
    assert _lib.load().ep_last_error().startswith(b"ep_route:")
