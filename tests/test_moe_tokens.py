"""The layer for a few tokens against a 64-bit reference."""
import ctypes

import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_util import U, gen, quantize_weight, randn, silu64, weight64

gpu = pytest.mark.gpu


def weights(E, H, I, kind, g):
    w13, w2 = randn((E, 2 * I, H), g) * H ** -0.5, randn((E, H, I), g) * I ** -0.5
    if kind == "bf16":
        return w13.to(torch.bfloat16), None, w2.to(torch.bfloat16), None
    a, b = quantize_weight(w13), quantize_weight(w2)
    return a[0], a[1], b[0], b[1]


def reference(x, idx, v, w):
    """(out, bound).  Both sums run in fp32 in another order: (terms / 32 + 24) * 2^-23 of the sum of the magnitudes,
    an element of x far below its block's largest is off by up to 2^-21 of that; h enters the second product to 2^-13
    of itself, or 2^-23 of its largest; bf16 rounding is held to 2^-8."""
    w13, s13, w2, s2 = w
    T, H = x.shape
    I = w2.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    X = x.double()
    for t in range(T):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if e < 0 or e >= w13.shape[0]:
                continue
            a = weight64(w13[e], None if s13 is None else s13[e])
            b = weight64(w2[e], None if s2 is None else s2[e])
            y, m = a @ X[t], (H / 32 + 24) * U * (a.abs() @ X[t].abs())
            m = m + 2.0 ** -21 * X[t].abs().max() * a.abs() @ (X[t].abs() < 2.0 ** -13 * X[t].abs().max()).double()
            h = silu64(y[:I]) * y[I:]
            dh = 1.1 * m[:I] * y[I:].abs() + silu64(y[:I]).abs() * m[I:] + 2.0 ** -13 * h.abs() + 2.0 ** -23 * h.abs().max()
            f = float(v[t, k])
            out[t] += f * (b @ h)
            err[t] += abs(f) * (b.abs() @ dh + (I / 32 + 24 + 64) * U * (b.abs() @ h.abs()))
    return out, err


def routing(T, E, K, g, mask=0.0):
    idx = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices
    idx = torch.where(torch.rand(T, K, generator=g, device="cuda") < mask, -1, idx)
    return idx.contiguous(), torch.rand(T, K, generator=g, device="cuda")


def check(x, idx, v, w, **kw):
    st = ep.new_status()
    out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], status=st, **kw)
    ep.check_status(st)
    ref, err = reference(x, idx, v, w)
    lim = 2.0 ** -8 * ref.abs() + err + 1e-38
    d = (out.double() - ref).abs()
    assert (d <= lim).all(), f"worst {float((d / lim).max()):.3g} of the bound"
    return out


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("T,E,K,H,I", [(1, 8, 2, 128, 128), (1, 1, 1, 128, 256), (3, 16, 4, 256, 128), (9, 4, 2, 384, 256),
                                       (17, 3, 3, 128, 384), (33, 2, 1, 256, 128), (64, 2, 2, 128, 128), (64, 64, 8, 256, 128),
                                       (5, 300, 6, 640, 128), (2, 8, 8, 1152, 1408)])
def test_layer(kind, T, E, K, H, I):
    g = gen(T * 1000 + E)
    idx, v = routing(T, E, K, g, mask=0.2 if T > 4 else 0.0)
    check(randn((T, H), g).to(torch.bfloat16), idx, v, weights(E, H, I, kind, g))


@gpu
@pytest.mark.parametrize("T,K,E", [(16, 2, 3), (4, 8, 4), (3, 10, 2), (1, 32, 64), (16, 2, 1), (17, 1, 2), (11, 3, 3), (2, 16, 5)])
def test_short_and_long_lists_with_repeats(T, K, E):
    """Up to 32 pairs one warp builds the expert list, beyond that the block does: repeats, masks, full entries."""
    g = gen(T * K + E)
    w = weights(E, 128, 128, "fp8", g)
    idx = torch.randint(-1, E, (T, K), generator=g, device="cuda")
    idx[0, 0] = E - 1
    check(randn((T, 128), g).to(torch.bfloat16), idx, torch.rand(T, K, generator=g, device="cuda"), w)


@gpu
@pytest.mark.parametrize("H,I", [(32, 32), (96, 160), (1056, 32), (64, 1120)])
def test_bf16_sizes_off_128(H, I):
    g = gen(H + I)
    idx, v = routing(11, 6, 3, g, mask=0.1)
    check(randn((11, H), g).to(torch.bfloat16), idx, v, weights(6, H, I, "bf16", g))


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_empty_tokens_and_all_masked(kind):
    g = gen(4)
    w = weights(6, 256, 128, kind, g)
    x = randn((12, 256), g).to(torch.bfloat16)
    idx, v = routing(12, 6, 3, g)
    idx[2] = idx[11] = -1
    x[2] = float("nan")                  # a token that nobody reads
    out = check(x, idx, v, w)
    assert (out[2].view(torch.int16) == 0).all() and (out[11].view(torch.int16) == 0).all()
    idx[:] = -1
    out = torch.full((12, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], out=out)
    assert (out.view(torch.int16) == 0).all()
    assert ep.moe_tokens(x[:0], idx[:0], v[:0], w[0], w[2], w[1], w[3]).shape == (0, 256)


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_repeated_experts_strides_and_workspace(kind):
    """A token may name an expert twice; x and out may be rows of wider arrays; a kept workspace needs no clearing."""
    g = gen(6)
    w = weights(5, 256, 256, kind, g)
    wide = randn((20, 264), g).to(torch.bfloat16)
    x = wide[:, 8:]
    x = torch.as_strided(wide, (20, 256), (264, 1), 0)
    idx = torch.randint(0, 5, (20, 4), generator=g, device="cuda")
    v = torch.rand(20, 4, generator=g, device="cuda")
    ws = torch.full((ep.moe_tokens_workspace(20, 4, 5, 256, 256, kind == "fp8"),), 0xAB, dtype=torch.uint8, device="cuda")
    obuf = torch.full((20, 300), 3.0, dtype=torch.bfloat16, device="cuda")
    out = check(x, idx, v, w, out=obuf[:, 7:263], workspace=ws)
    first = out.clone()
    assert (obuf[:, :7] == 3.0).all() and (obuf[:, 263:] == 3.0).all()
    for _ in range(3):                   # equal bits, whatever the workspace holds
        again = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], workspace=ws)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


@gpu
def test_non_finite_values_stay_with_their_token():
    g = gen(12)
    w = weights(4, 256, 128, "fp8", g)
    x = randn((10, 256), g).to(torch.bfloat16)
    idx, v = routing(10, 4, 2, g)
    clean = check(x, idx, v, w)
    x[3, 5], x[7, 0] = float("inf"), float("nan")
    out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3])
    ok = [t for t in range(10) if t not in (3, 7)]
    assert torch.equal(out[ok].view(torch.int16), clean[ok].view(torch.int16))
    assert not torch.isfinite(out[3]).any() and torch.isnan(out[7]).all()


@gpu
def test_entries_outside_the_experts_are_skipped_and_flagged():
    g = gen(13)
    w = weights(4, 128, 128, "fp8", g)
    x = randn((6, 128), g).to(torch.bfloat16)
    idx, v = routing(6, 4, 2, g)
    idx[1, 0], idx[4, 1] = 4, -2
    st = ep.new_status()
    out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], status=st)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(st)
    assert e.value.status == "EP_ERR_INVALID_INPUT"
    ref, err = reference(x, idx, v, w)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + err).all()


@gpu
def test_graph_and_side_stream():
    g = gen(14)
    w = weights(16, 512, 256, "fp8", g)
    x = randn((4, 512), g).to(torch.bfloat16)
    idx, v = routing(4, 16, 4, g)
    ws = torch.empty(ep.moe_tokens_workspace(4, 4, 16, 512, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty(4, 512, dtype=torch.bfloat16, device="cuda")
    call = lambda: ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], out=out, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(randn((4, 512), g).to(torch.bfloat16))
    out.zero_()
    graph.replay()
    ref, err = reference(x, idx, v, w)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + err).all()


@gpu
@pytest.mark.parametrize("kind,T,E,K,H,I", [("fp8", 18, 40, 2, 384, 128), ("fp8", 64, 3, 3, 128, 640), ("fp8", 64, 5, 1, 1152, 128),
                                            ("bf16", 40, 3, 3, 96, 160), ("bf16", 64, 4, 4, 1056, 32), ("bf16", 17, 1, 1, 32, 1120),
                                            ("bf16", 36, 6, 1, 64, 96), ("bf16", 35, 6, 1, 64, 96)])
def test_tokens_converted_beforehand(kind, T, E, K, H, I):
    """Above 16 tokens: pieces made once for all blocks; a token without an expert, one with a NaN, an infinity."""
    g = gen(T + E + H)
    w = weights(E, H, I, kind, g)
    x = randn((T, H), g).to(torch.bfloat16)
    idx, v = routing(T, E, K, g, mask=0.15)
    idx[0] = -1
    clean = check(x, idx, v, w)
    x[0] = float("nan")                  # nobody reads it
    x[2, 7], x[T - 1, H - 1] = float("inf"), float("nan")
    out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3])
    ok = [t for t in range(T) if t not in (2, T - 1) or (idx[t] < 0).all()]
    assert torch.equal(out[ok].view(torch.int16), clean[ok].view(torch.int16))
    for t in (2, T - 1):
        assert t in ok or not torch.isfinite(out[t]).any()
    idx[:] = -1
    assert (ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3]).view(torch.int16) == 0).all()


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_calls_of_all_lengths_share_a_workspace(kind):
    """Back to back on one stream, without a wait: each kernel starts while the one before drains."""
    g = gen(91)
    w = weights(4, 256, 256, kind, g)
    ws = torch.empty(max(ep.moe_tokens_workspace(t, 2, 4, 256, 256, kind == "fp8") for t in (1, 16, 17, 64)), dtype=torch.uint8, device="cuda")
    calls = []
    for t in (64, 1, 17, 16, 64, 64, 2, 33):
        x = randn((t, 256), g).to(torch.bfloat16)
        calls.append((x, *routing(t, 4, 2, g, mask=0.1)))
    outs = [ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], workspace=ws) for x, idx, v in calls]
    for (x, idx, v), out in zip(calls, outs):
        ref, err = reference(x, idx, v, w)
        assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + err + 1e-38).all()


@gpu
def test_refusals():
    g = gen(15)
    w13, s13, w2, s2 = weights(4, 256, 128, "fp8", g)
    x = randn((3, 256), g).to(torch.bfloat16)
    idx, v = routing(3, 4, 2, g)
    bad = [
        lambda: ep.moe_tokens(x.float(), idx, v, w13, w2, s13, s2),
        lambda: ep.moe_tokens(x.cpu(), idx, v, w13, w2, s13, s2),
        lambda: ep.moe_tokens(x, idx.int(), v, w13, w2, s13, s2),
        lambda: ep.moe_tokens(x, idx, v[:2], w13, w2, s13, s2),
        lambda: ep.moe_tokens(x, idx, v, w13, w2, s13, None),
        lambda: ep.moe_tokens(x, idx, v, w13, w2),
        lambda: ep.moe_tokens(x, idx, v, w13, w2.transpose(1, 2).contiguous(), s13, s2),
        lambda: ep.moe_tokens(x, idx, v, w13, w2, s13[:, :1].contiguous(), s2),
        lambda: ep.moe_tokens(x, idx, v, w13, w2, s13, s2, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: ep.moe_tokens(x.repeat(30, 1), idx.repeat(30, 1), v.repeat(30, 1), w13, w2, s13, s2),   # 90 tokens
        lambda: ep.moe_tokens(x, idx, v, w13, w2, s13, s2, out=torch.empty(3, 255, dtype=torch.bfloat16, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, ep.EpError)):
            f()
            pytest.fail(f"refusal {i} was accepted")


def test_c_refusals_without_a_gpu():
    from combine_get_dispatch_histograms_gb300 import _lib
    lib = _lib.load()
    names = ("w13", "w13_scales", "w2", "w2_scales", "experts", "hidden", "inter")
    good = dict(w13=256, w13_scales=256, w2=256, w2_scales=256, experts=4, hidden=128, inter=128)
    call = lambda T=1, K=1, x=256, **k: lib.ep_moe_tokens(  # noqa: E731
        x, 1024, T, 256, 256, K, ctypes.byref(_lib.EpMoeWeights(*[dict(good, **k)[n] for n in names])), 256, 1024, 256, 0,
        None, None)
    assert call(T=0) == 0
    for bad in (dict(T=65), dict(T=-1), dict(K=0), dict(K=33), dict(experts=0), dict(experts=5000), dict(hidden=96), dict(inter=64),
                dict(w2_scales=None), dict(w13=None), dict(w13=264), dict(x=264)):
        assert call(**bad) == -1, bad
    size = lambda T, **k: lib.ep_moe_tokens_workspace(  # noqa: E731
        T, 1, ctypes.byref(_lib.EpMoeWeights(*[dict(good, **k)[n] for n in names])))
    assert size(65) == 0 and size(1, hidden=0) == 0 and lib.ep_moe_tokens_workspace(1, 1, None) == 0


@gpu
def test_a_workspace_with_gaps_is_refused():
    """It would be written as if it had none."""
    g = gen(16)
    w13, s13, w2, s2 = weights(4, 256, 128, "fp8", g)
    x = randn((3, 256), g).to(torch.bfloat16)
    idx, v = routing(3, 4, 2, g)
    need = ep.moe_tokens_workspace(3, 2, 4, 256, 128)
    buf = torch.full((2 * need,), 0xAB, dtype=torch.uint8, device="cuda")
    for ws in (buf[::2], buf.view(-1, 32)[:, :16]):
        assert ws.nbytes >= need
        with pytest.raises(ValueError, match="contiguous"):
            ep.moe_tokens(x, idx, v, w13, w2, s13, s2, workspace=ws)
    assert (buf == 0xAB).all()


@pytest.mark.parametrize("bad", [dict(T=65), dict(T=0), dict(T=-1), dict(K=0), dict(K=33), dict(experts=0), dict(experts=4097),
                                 dict(hidden=96), dict(hidden=160), dict(inter=64), dict(inter=-128), dict(w2_scales=None),
                                 dict(hidden=1 << 29), dict(inter=1 << 30), dict(w13_scales=None, w2_scales=None, hidden=48),
                                 dict(w13_scales=None, w2_scales=None, inter=16)])
def test_refused_sizes_need_no_workspace(bad):
    """What ep_moe_tokens refuses has a workspace of 0 bytes."""
    from combine_get_dispatch_histograms_gb300 import _lib
    lib = _lib.load()
    c = dict(dict(T=1, K=1, w13=256, w13_scales=256, w2=256, w2_scales=256, experts=4, hidden=128, inter=128), **bad)
    w = _lib.EpMoeWeights(*[c[n] for n in ("w13", "w13_scales", "w2", "w2_scales", "experts", "hidden", "inter")])
    call = lib.ep_moe_tokens(256, 1 << 32, c["T"], 256, 256, c["K"], ctypes.byref(w), 256, 1 << 32, 256, 0, None, None)
    assert call == (0 if c["T"] == 0 else -1)
    assert lib.ep_moe_tokens_workspace(c["T"], c["K"], ctypes.byref(w)) == 0


@gpu
def test_every_refused_size_needs_no_workspace_on_a_gpu():
    """The same where the device is known, next to sizes that are taken."""
    size = lambda T=1, K=1, E=4, H=128, I=128, fp8=True: ep.moe_tokens_workspace(T, K, E, H, I, fp8)  # noqa: E731
    assert size() > 0 and size(fp8=False, H=32, I=160) > 0 and size(T=64, K=32, E=4096) > 0
    for bad in (dict(T=65), dict(T=0), dict(K=33), dict(E=4097), dict(H=160), dict(I=64), dict(H=48, fp8=False), dict(H=1 << 29)):
        assert size(**bad) == 0, bad


@pytest.mark.parametrize("bad", ["topk_idx", "topk_weights", "out", "w13_scales", "w2_scales", "status"])
def test_c_refuses_pointers_off_their_elements(bad):
    from combine_get_dispatch_histograms_gb300 import _lib
    lib = _lib.load()
    at = {n: 256 + (1 if n == bad else 0) for n in ("topk_idx", "topk_weights", "out", "w13_scales", "w2_scales", "status")}
    if bad == "topk_idx":
        at[bad] = 260                    # a multiple of 4, not of 8
    w = _lib.EpMoeWeights(256, at["w13_scales"], 256, at["w2_scales"], 4, 128, 128)
    assert lib.ep_moe_tokens(256, 128, 1, at["topk_idx"], at["topk_weights"], 1, ctypes.byref(w), at["out"], 128, 256, 1 << 30,
                             at["status"], None) == -1
    assert b"aligned to its elements" in lib.ep_last_error()


@gpu
@pytest.mark.parametrize("T,K", [(1, 8), (4, 8), (5, 7), (16, 3), (15, 8)])
def test_few_tokens_of_a_large_layer(T, K):
    """100 MB of weights: the pieces are made beforehand for fewer than 17 tokens too, with short and long lists."""
    from expert_shapes import launches
    E, H, I = 12, 2048, 2176
    g = gen(T * 10 + K)
    w = weights(E, H, I, "fp8", g)
    x = randn((T, H), g).to(torch.bfloat16)
    idx, v = routing(T, E, K, g, mask=0.1 if T > 1 else 0.0)
    out, ws = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(
        ep.moe_tokens_workspace(T, K, E, H, I), dtype=torch.uint8, device="cuda")
    names = [n for n, _ in launches(lambda s: ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3], out=out, workspace=ws, stream=s))]
    assert ["form_kernel" in n for n in names] == [True, False, True, False], names
    clean = check(x, idx, v, w)
    if T > 1:
        x[0, 3] = float("nan")
        out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3])
        assert torch.isnan(out[0]).all() or (idx[0] < 0).all()
        assert torch.equal(out[1:].view(torch.int16), clean[1:].view(torch.int16))
        idx[1] = -1                      # other routing, another order of the sums
        out = ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3])
        assert (out[1].view(torch.int16) == 0).all()
        x[0] = 1.0
        check(x, idx, v, w)
    idx[:] = -1
    assert (ep.moe_tokens(x, idx, v, w[0], w[2], w[1], w[3]).view(torch.int16) == 0).all()
