"""A NaN or an infinity of the rows or weights reaches every output that reads it, and no other."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_shapes import form_of
from expert_util import assert_fp8_close, gen, quantize_rows, quantize_weight, randn, rows64, swiglu64, weight64

gpu = pytest.mark.gpu

#                form: groups, rows of each, K, I, expected rows
FORMS = {"one": (40, 60, 256, 512, 64), "pairs": (40, 300, 256, 512, 500), "cluster": (2, 70, 1024, 256, 0)}


def case(form, seed):
    G, m, K, I, expected = FORMS[form]
    g = gen(seed)
    x, xs = quantize_rows(randn((G * m, K), g))
    w, ws = quantize_weight(randn((G, 2 * I, K), g) * K ** -0.5)
    assert form_of(G * m, G, 2 * I, K, expected) == form
    kw = dict(counts=torch.full((G,), m, dtype=torch.int32, device="cuda"),
              offsets=torch.arange(0, G * m, m, dtype=torch.int32, device="cuda"), expected_rows=expected)
    return x, xs, w, ws, kw, (G, m, K, I)


def nan_blocks(codes, scales):
    """[rows][I / 128]: every value that the block stands for is NaN."""
    return torch.isnan(rows64(codes, scales)).view(codes.shape[0], -1, 128).all(-1)


def clean_rows_hold(codes, scales, x, xs, w, ws, G, m, bad):
    for e in range(G):
        r = torch.arange(e * m, e * m + m, device="cuda")
        r = r[~bad[r]]
        assert_fp8_close(codes[r], scales[r], *swiglu64(rows64(x[r], xs[r]), weight64(w[e], ws[e])), f"group {e}")


@gpu
@pytest.mark.parametrize("form", FORMS)
def test_swiglu_keeps_a_rows_nan(form):
    """A NaN code, a NaN scale and an infinite one make all of their row NaN, codes and scales, and what reads them."""
    x, xs, w, ws, kw, (G, m, K, I) = case(form, 31)
    rows = x.shape[0]
    x[3, 7], x[rows - 1, K - 1] = 0x7F, 0xFF
    xs[m, 1], xs[m + 40, 0] = float("nan"), float("inf")
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[3, rows - 1, m, m + 40]] = True
    codes, scales = ep.expert_swiglu(x, xs, w, ws, **kw)
    assert torch.isnan(scales[bad]).all() and nan_blocks(codes, scales)[bad].all()
    assert torch.isfinite(scales[~bad]).all()
    clean_rows_hold(codes, scales, x, xs, w, ws, G, m, bad)
    w2, w2s = quantize_weight(randn((G, 136, I), gen(32)) * I ** -0.5)
    y = ep.expert_gemm(codes, scales, w2, w2s, **kw)
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("half", ["gate", "up"])
def test_swiglu_keeps_a_weights_nan(form, half):
    """A NaN code of the weight makes its block of 128 output channels NaN, in the rows of its expert."""
    x, xs, w, ws, kw, (G, m, K, I) = case(form, 33)
    clean = ep.expert_swiglu(x, xs, w, ws, **kw)
    w[1, (0 if half == "gate" else I) + 130, 5] = 0x7F           # channel 130: block 1
    codes, scales = ep.expert_swiglu(x, xs, w, ws, **kw)
    want = torch.zeros(G * m, I // 128, dtype=torch.bool, device="cuda")
    want[m:2 * m, 1] = True
    assert torch.equal(torch.isnan(scales), want) and torch.equal(nan_blocks(codes, scales), want)
    keep = (~want).repeat_interleave(128, 1)
    assert torch.equal(codes[keep], clean[0][keep]) and torch.equal(scales[~want], clean[1][~want])
