"""Each block (or pair) of the product kernel makes many tiles: what is carried from one to the next."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_shapes import form_of, tiles_of
from expert_util import assert_bf16_close, assert_fp8_close, gen, product64, quantize_rows, quantize_weight, randn, rows64, swiglu64, weight64

gpu = pytest.mark.gpu

RAGGED = [0, 1, 31, 128, 129, 255, 256, 257, 300, 513, 64, 0, 640, 127, 2, 384] * 4
CHUNKED = [4500, 0, 1, 2049, 300, 6200, 128]      # groups of more rows than share a pass over the weight's tiles
FORMS = {"one": 64, "pairs": 500}


def case(counts, K, N, seed, gap=1):
    g = gen(seed)
    off, r = [], 0
    for c in counts:
        off.append(r + gap)
        r += gap + c
    x, xs = quantize_rows(randn((r, K), g))
    w, ws = quantize_weight(randn((len(counts), N, K), g) * K ** -0.5)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(counts), i32(off), off, x, xs, w, ws


def owned(counts, off, rows):
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for o, c in zip(off, counts):
        own[o:o + c] = True
    return own


def many(counts, N, rows, K, form, least=6):
    assert form_of(rows, len(counts), N, K, FORMS[form]) == form
    tiles, units = tiles_of(counts, N, form)
    assert tiles >= least * units, f"{tiles} tiles for {units}"


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("KB", [1, 2, 3, 5, 9, 12])
@pytest.mark.parametrize("N,stride", [(2048, 2048), (2043, 2043), (2040, 2048), (2043, 2048)])
def test_gemm(form, KB, N, stride):
    K = 128 * KB
    cnt, off, hoff, x, xs, w, ws = case(RAGGED, K, N, seed=KB + N)
    many(RAGGED, N, x.shape[0], K, form)
    wide = torch.full((x.shape[0], stride), 7.0, dtype=torch.bfloat16, device="cuda")
    st = ep.new_status()
    for _ in range(2):                   # back to back: the second starts while the first drains
        ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=wide[:, :N], expected_rows=FORMS[form], status=st)
    ep.check_status(st)
    for e, (o, c) in enumerate(zip(hoff, RAGGED)):
        if c:
            assert_bf16_close(wide[o:o + c, :N], *product64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])), f"group {e}")
    assert (wide[~owned(RAGGED, hoff, x.shape[0])] == 7.0).all() and (wide[:, N:] == 7.0).all()


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("KB", [1, 2, 3, 5, 9, 12])
def test_swiglu(form, KB):
    K, I = 128 * KB, 1024
    cnt, off, hoff, x, xs, w, ws = case(RAGGED, K, 2 * I, seed=KB)
    many(RAGGED, 2 * I, x.shape[0], K, form)
    codes = torch.full((x.shape[0], I), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((x.shape[0], I // 128), 5.0, device="cuda")
    st = ep.new_status()
    for _ in range(2):
        ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, out=(codes, scales), expected_rows=FORMS[form], status=st)
    ep.check_status(st)
    for e, (o, c) in enumerate(zip(hoff, RAGGED)):
        if c:
            h, err = swiglu64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e]))
            assert_fp8_close(codes[o:o + c], scales[o:o + c], h, err, f"group {e}")
    rest = ~owned(RAGGED, hoff, x.shape[0])
    assert (codes[rest] == 9).all() and (scales[rest] == 5.0).all()


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("KB", [1, 5])
def test_groups_of_several_chunks_of_rows(form, KB):
    K, N = 128 * KB, 1792
    cnt, off, hoff, x, xs, w, ws = case(CHUNKED, K, N, seed=KB)
    many(CHUNKED, N, x.shape[0], K, form, least=4)
    out = torch.full((x.shape[0], N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, expected_rows=FORMS[form])
    codes, scales = ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=FORMS[form])
    for e, (o, c) in enumerate(zip(hoff, CHUNKED)):
        if c:
            X, W = rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])
            assert_bf16_close(out[o:o + c], *product64(X, W), f"group {e}")
            assert_fp8_close(codes[o:o + c], scales[o:o + c], *swiglu64(X, W), f"group {e}")
    assert (out[~owned(CHUNKED, hoff, x.shape[0])] == 7.0).all()


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("KB,N", [(5, 5120), (11, 4608)])
def test_rest_of_the_ring_in_both_forms(form, KB, N):
    """KB odd and above the ring's four stages, groups of one tile to three."""
    counts, K = [300, 0, 513, 256, 1, 255, 640], 128 * KB
    cnt, off, hoff, x, xs, w, ws = case(counts, K, N, seed=KB)
    assert form_of(x.shape[0], len(counts), N, K, FORMS[form]) == form
    out = ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=FORMS[form])
    codes, scales = ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=FORMS[form])
    for e, (o, c) in enumerate(zip(hoff, counts)):
        if c:
            X, W = rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])
            assert_bf16_close(out[o:o + c], *product64(X, W), f"group {e}")
            assert_fp8_close(codes[o:o + c], scales[o:o + c], *swiglu64(X, W), f"group {e}")


@gpu
def test_short_launches_of_both_forms_in_turn():
    """Blocks end and start on the same SM by the hundred: nothing that one launch signals arrives in the next."""
    counts = [130, 200, 256] * 28
    cnt, off, hoff, x, xs, w, ws = case(counts, 128, 256, seed=77)
    outs, forms = {}, ("pairs", "one", "pairs", "pairs", "one")
    for form in ("one", "pairs"):
        assert form_of(x.shape[0], len(counts), 256, 128, FORMS[form]) == form
        outs[form] = ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=FORMS[form])
        for e, (o, c) in enumerate(zip(hoff, counts)):
            assert_bf16_close(outs[form][o:o + c], *product64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])), f"group {e}")
    own = owned(counts, hoff, x.shape[0])
    st = ep.new_status()
    got = [ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=FORMS[f], status=st) for f in forms * 60]
    ep.check_status(st)
    for f, y in zip(forms * 60, got):
        assert torch.equal(y[own].view(torch.int16), outs[f][own].view(torch.int16))
