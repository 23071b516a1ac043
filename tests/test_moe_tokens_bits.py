"""moe_tokens holds x and h in no fewer bits than a 32-bit form: sums in which they cancel."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_util import U, gen, silu64, weight64

gpu = pytest.mark.gpu


def ints(shape, g, top):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").float()


def layer(kind, w13, s13, w2, s2):
    """Weights that are integers times a power of two per block of 128 x 128, both exact in e4m3 and in bf16."""
    if kind == "fp8":
        code = lambda w: w.to(torch.float8_e4m3fn)  # noqa: E731
        return code(w13), s13, code(w2), s2
    spread = lambda w, s: (w * s.repeat_interleave(128, 1).repeat_interleave(128, 2)).to(torch.bfloat16)  # noqa: E731
    return spread(w13, s13), None, spread(w2, s2), None


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 64])
def test_h_that_cancels(kind, T):
    """Channels 2i and 2i + 1 of h differ by about 2^-15 of themselves, and an output is one minus the other.

    x and the weights are integers times powers of two, so that gate and up are exact in fp32, and an output adds two
    products.  What rounds: silu and its product with up (2^-20 of h, of both), h itself and the sum of its two products
    (2^-21 together, of both; for an element far below its 128 channels' largest 2^-37 of that), and the output."""
    g = gen(41 + T)
    H, I, E = 256, 256, 2
    x = ints((T, H), g, 2)
    x[:, 0] = 1
    w13 = torch.zeros(E, 2 * I, H, device="cuda")
    w13[:, 0:I:2] = ints((E, I // 2, H), g, 2)
    w13[:, 1:I:2] = w13[:, 0:I:2]                          # the same gate
    w13[:, I::2] = ints((E, I // 2, H), g, 2)
    w13[:, I + 1::2] = w13[:, I::2]
    w13[:, I + 1::2, 128:] = ints((E, I // 2, 128), g, 2)  # up differs in the second block, whose scale is small
    s13 = torch.full((E, 2 * I // 128, 2), 2.0 ** -5, device="cuda")
    s13[:, :, 1] = 2.0 ** -20
    w2 = torch.zeros(E, H, I, device="cuda")
    out_ch = torch.arange(H, device="cuda")
    pair = (out_ch * 37 + 11) % (I // 2)
    w2[:, out_ch, 2 * pair], w2[:, out_ch, 2 * pair + 1] = 1, -1
    s2 = torch.ones(E, H // 128, I // 128, device="cuda")
    w = layer(kind, w13, s13, w2, s2)
    idx = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    v = torch.ones(T, 1, device="cuda")
    xb = x.to(torch.bfloat16)
    out = ep.moe_tokens(xb, idx, v, w[0], w[2], w[1], w[3]).double()
    for t in range(T):
        e = int(idx[t, 0])
        y = weight64(w[0][e], None if w[1] is None else w[1][e]) @ xb[t].double()
        assert (y == y.float().double()).all()
        h = silu64(y[:I]) * y[I:]
        a, b = h[2 * pair], h[2 * pair + 1]
        top = h.view(-1, 128).abs().amax(1)[2 * pair // 128]
        lim = 2.0 ** -8 * (a - b).abs() + (2.0 ** -20 + 2.0 ** -21) * (a.abs() + b.abs()) + 2 * 2.0 ** -37 * top + 1e-38
        d = (out[t] - (a - b)).abs()
        assert (d <= lim).all(), f"token {t}: {int((d > lim).sum())} outputs, worst {float((d / lim).max()):.3g} of the bound"


@gpu
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 16, 17, 40])
@pytest.mark.parametrize("power", [12, 18, 26])
def test_x_beside_an_outlier(kind, T, power):
    """One channel of x is 2^power times the others and no weight reads it: the others count in full.

    The bound is that of fp32 sums in another order, as for any x: (terms / 32 + 24) * 2^-23 of the sum of the magnitudes."""
    g = gen(53 + T)
    H, I, E = 256, 128, 3
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, 77] = 2.0 ** power
    x[:, 200] = -(2.0 ** power)
    xb = x.to(torch.bfloat16)
    w13 = ints((E, 2 * I, H), g, 8)
    w13[:, :, 77] = w13[:, :, 200] = 0
    w2 = ints((E, H, I), g, 8)
    s13, s2 = torch.full((E, 2, 2), 2.0 ** -6, device="cuda"), torch.full((E, 2, 1), 2.0 ** -5, device="cuda")
    w = layer(kind, w13, s13, w2, s2)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:2] for _ in range(T)])
    v = torch.rand(T, 2, generator=g, device="cuda")
    out = ep.moe_tokens(xb, idx, v, w[0], w[2], w[1], w[3]).double()
    for t in range(T):
        ref = torch.zeros(H, dtype=torch.float64, device="cuda")
        err = torch.zeros_like(ref)
        for k in range(2):
            e, f = int(idx[t, k]), float(v[t, k])
            a, b = (weight64(w[i][e], None if w[i + 1] is None else w[i + 1][e]) for i in (0, 2))
            X = xb[t].double()
            y, m = a @ X, (H / 32 + 24) * U * (a.abs() @ X.abs())
            h = silu64(y[:I]) * y[I:]
            dh = 1.1 * m[:I] * y[I:].abs() + silu64(y[:I]).abs() * m[I:] + 1.1 * m[:I] * m[I:] + 2.0 ** -20 * h.abs()
            ref += f * (b @ h)
            err += f * (b.abs() @ dh + (I / 32 + 24) * U * (b.abs() @ h.abs()))
        lim = 2.0 ** -8 * ref.abs() + err
        d = (out[t] - ref).abs()
        assert (d <= lim).all(), f"token {t}: worst {float((d / lim).max()):.3g} of the bound"
