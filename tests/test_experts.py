"""The expert products (FP8 rows x FP8 weights) against 64-bit references."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_util import (assert_bf16_close, assert_fp8_close, gen, product64, quantize_rows, quantize_weight, randn,
                               rows64, swiglu64, weight64)

gpu = pytest.mark.gpu


def groups_of(counts, gap=0):
    """(counts, offsets, rows) on the GPU; `gap` unused rows before every group."""
    off, r = [], 0
    for c in counts:
        r += gap
        off.append(r)
        r += c
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(counts), i32(off), off, max(1, r)


def case(counts, K, N, seed=0, gap=0):
    g = gen(seed)
    cnt, off, hoff, rows = groups_of(counts, gap)
    x, xs = quantize_rows(randn((rows, K), g))
    w, ws = quantize_weight(randn((len(counts), N, K), g) * K ** -0.5)
    return cnt, off, hoff, x, xs, w, ws


RAGGED = [0, 1, 7, 128, 129, 31, 0, 255, 300, 0]
LONG = [300, 0, 513, 256, 1, 255, 640]   # long groups: pairs of blocks, with full, half-full and one-row tiles


@gpu
@pytest.mark.parametrize("K,N", [(128, 128), (128, 1), (256, 130), (640, 256), (1408, 600), (2048, 1099), (512, 8), (384, 257)])
@pytest.mark.parametrize("counts", [[1], [5, 0, 64], RAGGED, LONG])
def test_gemm_ragged(K, N, counts):
    cnt, off, hoff, x, xs, w, ws = case(counts, K, N, seed=K + N, gap=3)
    st = ep.new_status()
    out = torch.full((x.shape[0], N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, status=st)
    ep.check_status(st)
    own = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(hoff, counts)):
        own[o:o + c] = True
        if c:
            y, err = product64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e]))
            assert_bf16_close(out[o:o + c], y, err, f"group {e}")
    assert (out[~own] == 7.0).all(), "rows of no group were written"


@gpu
@pytest.mark.parametrize("K,I", [(128, 128), (640, 384), (1024, 256), (4096, 128)])
@pytest.mark.parametrize("counts", [[1], [5, 0, 64], RAGGED, LONG])
def test_swiglu_ragged(K, I, counts):
    cnt, off, hoff, x, xs, w, ws = case(counts, K, 2 * I, seed=K + I, gap=2)
    st = ep.new_status()
    codes = torch.full((x.shape[0], I), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((x.shape[0], I // 128), 5.0, device="cuda")
    ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, out=(codes, scales), status=st)
    ep.check_status(st)
    own = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(hoff, counts)):
        own[o:o + c] = True
        if c:
            h, err = swiglu64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e]))
            assert_fp8_close(codes[o:o + c], scales[o:o + c], h, err, f"group {e}")
    assert (codes[~own] == 9).all() and (scales[~own] == 5.0).all(), "rows of no group were written"


@gpu
@pytest.mark.parametrize("rows", [1, 2, 33, 127, 128, 129, 256, 500])
@pytest.mark.parametrize("K,N", [(2048, 512), (128, 77), (7168, 256)])
def test_gemm_dense(rows, K, N):
    g = gen(rows + K)
    x, xs = quantize_rows(randn((rows, K), g))
    w, ws = quantize_weight(randn((1, N, K), g) * K ** -0.5)
    out = ep.expert_gemm(x, xs, w[0], ws[0])
    y, err = product64(rows64(x, xs), weight64(w[0], ws[0]))
    assert_bf16_close(out, y, err)


@gpu
@pytest.mark.parametrize("rows", [1, 3, 130])
@pytest.mark.parametrize("K,I", [(7168, 128), (1408, 256), (512, 640)])
def test_swiglu_dense(rows, K, I):
    """Few tiles: the blocks of a cluster share K."""
    g = gen(rows + K + I)
    x, xs = quantize_rows(randn((rows, K), g))
    w, ws = quantize_weight(randn((1, 2 * I, K), g) * K ** -0.5)
    codes, scales = ep.expert_swiglu(x, xs, w[0], ws[0])
    assert_fp8_close(codes, scales, *swiglu64(rows64(x, xs), weight64(w[0], ws[0])))


@gpu
@pytest.mark.parametrize("K,N", [(4096, 136), (2560, 3000), (16384, 200), (5376, 7000), (6144, 4096), (6272, 9999), (768, 9728)])
def test_one_row_by_clusters_of_all_sizes(K, N):
    g = gen(K + N)
    q, s = quantize_rows(randn((3, K), g))
    w, ws = quantize_weight(randn((1, N, K), g) * K ** -0.5)
    for rows in (1, 3):
        assert_bf16_close(ep.expert_gemm(q[:rows], s[:rows], w[0], ws[0]), *product64(rows64(q[:rows], s[:rows]), weight64(w[0], ws[0])))
    if N % 256 == 0:
        codes, scales = ep.expert_swiglu(q, s, w[0], ws[0])
        assert_fp8_close(codes, scales, *swiglu64(rows64(q, s), weight64(w[0], ws[0])))


@gpu
@pytest.mark.parametrize("expected", [64, 200, 300, 500])
@pytest.mark.parametrize("K,N", [(128, 256), (640, 512), (1408, 768), (2048, 1280)])
def test_both_shapes_on_long_and_ragged_groups(K, N, expected):
    """One block a tile or two, whatever the groups hold."""
    for counts in (LONG, RAGGED):
        cnt, off, hoff, x, xs, w, ws = case(counts, K, N, seed=K + N + expected, gap=2)
        out = torch.full((x.shape[0], N), 7.0, dtype=torch.bfloat16, device="cuda")
        ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, expected_rows=expected)
        hc, hs = (torch.full((x.shape[0], n), 7, dtype=t, device="cuda") for n, t in ((N // 2, torch.uint8), (N // 256, torch.float32)))
        ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, out=(hc, hs), expected_rows=expected)
        own = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
        for e, (o, c) in enumerate(zip(hoff, counts)):
            own[o:o + c] = True
            if c:
                X, W = rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])
                assert_bf16_close(out[o:o + c], *product64(X, W), f"group {e}")
                assert_fp8_close(hc[o:o + c], hs[o:o + c], *swiglu64(X, W))
        assert (out[~own] == 7.0).all() and (hc[~own] == 7).all() and (hs[~own] == 7).all()


@gpu
@pytest.mark.parametrize("shift,stride", [(0, 576), (16, 576), (8, 576), (0, 568), (8, 568), (4, 568), (0, 571), (3, 571)])
def test_short_groups_at_every_alignment_of_the_output(shift, stride):
    """Stores of 32, 16 and 2 bytes; the elements between the rows keep their values."""
    counts = [60, 33, 0, 1] * 16        # more tiles than share their K
    cnt, off, hoff, x, xs, w, ws = case(counts, 256, 552, seed=shift + stride)
    buf = torch.full((x.shape[0] * stride + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(buf, (x.shape[0], 552), (stride, 1), shift)
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, expected_rows=1)
    for e, (o, c) in enumerate(zip(hoff, counts)):
        if c:
            assert_bf16_close(out[o:o + c], *product64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])), f"group {e}")
    buf[shift:shift + x.shape[0] * stride].view(-1, stride)[:, :552] = 9.0
    assert (buf == 9.0).all()


@gpu
@pytest.mark.parametrize("counts", [[0, 0, 3], [0, 0, 0], [130, 1, 0]])
def test_few_tiles_with_empty_groups(counts):
    cnt, off, hoff, x, xs, w, ws = case(counts, 1024, 136, seed=sum(counts), gap=1)
    out = torch.full((x.shape[0], 136), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out)
    own = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(hoff, counts)):
        own[o:o + c] = True
        if c:
            assert_bf16_close(out[o:o + c], *product64(rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])), f"group {e}")
    assert (out[~own] == 7.0).all()


@gpu
@pytest.mark.parametrize("fn", ["gemm", "swiglu"])
def test_packed_regions(fn):
    g = gen(3)
    E, cap, K, N = 6, 200, 384, 256
    counts = [0, 1, 200, 130, 17, 64]
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    x, xs = quantize_rows(randn((E, cap, K), g))
    w, ws = quantize_weight(randn((E, N, K), g) * K ** -0.5)
    if fn == "gemm":
        out = ep.expert_gemm(x, xs, w, ws, counts=cnt)
    else:
        codes, scales = ep.expert_swiglu(x, xs, w, ws, counts=cnt)
    for e, c in enumerate(counts):
        if not c:
            continue
        r, wt = rows64(x[e, :c], xs[e, :c]), weight64(w[e], ws[e])
        if fn == "gemm":
            assert_bf16_close(out[e, :c], *product64(r, wt), f"expert {e}")
        else:
            assert_fp8_close(codes[e, :c], scales[e, :c], *swiglu64(r, wt), f"expert {e}")


@gpu
@pytest.mark.parametrize("K,N", [(128, 128), (512, 200), (1024, 8)])
def test_gemm_exact_integers(K, N):
    """Small integers times powers of two: the sum is exact in fp32, so the result is the exact value rounded once."""
    g = gen(K * 3 + N)
    rows = 150
    v = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float()
    x = v.to(torch.float8_e4m3fn)
    xs = torch.exp2(torch.randint(-3, 4, (rows, K // 128), generator=g, device="cuda").float())
    wc = w.to(torch.float8_e4m3fn)
    ws = torch.exp2(torch.randint(-3, 4, (-(-N // 128), K // 128), generator=g, device="cuda").float())
    out = ep.expert_gemm(x, xs, wc, ws)
    ref = rows64(x, xs) @ weight64(wc, ws).t()
    assert (ref == ref.float().double()).all()
    assert torch.equal(out.view(torch.int16), ref.float().to(torch.bfloat16).view(torch.int16))


@gpu
def test_gemm_strides_and_unaligned_output():
    """Rows of the FP8 dispatch (scales behind the codes), an output inside a wider array, and one at an odd element."""
    g = gen(17)
    rows, K, N = 140, 256, 264
    q, s = quantize_rows(randn((rows, K), g))
    buf = torch.zeros(rows, K + 16, dtype=torch.uint8, device="cuda")
    buf[:, :K] = q
    buf[:, K:K + 8] = s.view(torch.uint8)
    x, xs = buf[:, :K], buf[:, K:K + 8].view(torch.float32)
    w, ws = quantize_weight(randn((1, N, K), g) * K ** -0.5)
    y, err = product64(rows64(q, s), weight64(w[0], ws[0]))
    for pad, first in ((24, 8), (7, 3)):
        wide = torch.full((rows, N + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        ep.expert_gemm(x, xs, w[0], ws[0], out=wide[:, first:first + N])
        assert_bf16_close(wide[:, first:first + N], y, err)
        assert (wide[:, :first] == 3.0).all() and (wide[:, first + N:] == 3.0).all()


@gpu
def test_swiglu_writes_fp8_rows_that_gemm_reads():
    """The two products chained through FP8 rows with their scales behind the codes, on a stream of their own."""
    g = gen(23)
    counts = [70, 0, 3, 140]
    cnt, off, hoff, x, xs, w13, w13s = case(counts, 256, 512, seed=23)
    w2, w2s = quantize_weight(randn((4, 300, 256), g) * 256 ** -0.5)
    rows = x.shape[0]
    buf = torch.zeros(rows, 256 + 16, dtype=torch.uint8, device="cuda")
    h, hs = buf[:, :256], buf[:, 256:264].view(torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ep.expert_swiglu(x, xs, w13, w13s, counts=cnt, offsets=off, out=(h, hs), stream=side)
    y = ep.expert_gemm(h, hs, w2, w2s, counts=cnt, offsets=off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for e, (o, c) in enumerate(zip(hoff, counts)):
        if c:
            assert_fp8_close(h[o:o + c], hs[o:o + c], *swiglu64(rows64(x[o:o + c], xs[o:o + c]), weight64(w13[e], w13s[e])))
            assert_bf16_close(y[o:o + c], *product64(rows64(h[o:o + c], hs[o:o + c]), weight64(w2[e], w2s[e])))


@gpu
def test_non_finite_and_zero_rows_stay_in_their_row():
    g = gen(29)
    rows, K, N = 160, 256, 512
    x, xs = quantize_rows(randn((rows, K), g))
    x[3, 7] = 0x7F                       # a NaN code
    xs[5, 1] = float("inf")
    x[9] = 0
    w, ws = quantize_weight(randn((1, N, K), g) * K ** -0.5)
    out = ep.expert_gemm(x, xs, w[0], ws[0])
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    ok[3] = ok[5] = False
    y, err = product64(rows64(x[ok], xs[ok]), weight64(w[0], ws[0]))
    assert_bf16_close(out[ok], y, err)
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[5]).any()
    codes, scales = ep.expert_swiglu(x, xs, w[0], ws[0])
    h, err = swiglu64(rows64(x[ok], xs[ok]), weight64(w[0], ws[0]))
    assert_fp8_close(codes[ok], scales[ok], h, err)
    assert (codes[9] & 0x7F == 0).all() and (scales[9] == 0).all()


@gpu
@pytest.mark.parametrize("expected", [1, 4096])
def test_expected_rows_only_choose_the_shape(expected):
    """Both shapes of the kernel on the same groups, whatever the caller expects."""
    for counts in (RAGGED, LONG):
        cnt, off, hoff, x, xs, w, ws = case(counts, 384, 512, seed=sum(counts))
        y = ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=expected)
        codes, scales = ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, expected_rows=expected)
        for e, (o, c) in enumerate(zip(hoff, counts)):
            if c:
                r, wt = rows64(x[o:o + c], xs[o:o + c]), weight64(w[e], ws[e])
                assert_bf16_close(y[o:o + c], *product64(r, wt), f"group {e}")
                assert_fp8_close(codes[o:o + c], scales[o:o + c], *swiglu64(r, wt), f"group {e}")


@gpu
def test_repeats_bitwise():
    cnt, off, _, x, xs, w, ws = case(RAGGED, 1024, 512, seed=5)
    a = ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=torch.zeros(x.shape[0], 512, dtype=torch.bfloat16, device="cuda"))
    for _ in range(3):
        b = ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=torch.zeros_like(a))
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@gpu
def test_rows_outside_the_arrays_are_cut_and_flagged():
    cnt, off, hoff, x, xs, w, ws = case([40, 50], 128, 256, seed=8)
    st = ep.new_status()
    off = off.clone()
    off[1] = 60                          # rows 60 .. 109 of 90
    out = torch.zeros(90, 256, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, status=st)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(st)
    assert e.value.status == "EP_ERR_CAPACITY"
    ep.check_status(st)                  # cleared
    for g_, (o, n) in enumerate(((0, 40), (60, 30))):
        assert_bf16_close(out[o:o + n], *product64(rows64(x[o:o + n], xs[o:o + n]), weight64(w[g_], ws[g_])))


@gpu
def test_refusals():
    cnt, off, _, x, xs, w, ws = case([4, 4], 256, 256, seed=9)
    ok = dict(counts=cnt, offsets=off)
    bad = [
        lambda: ep.expert_gemm(x.cpu(), xs, w, ws, **ok),
        lambda: ep.expert_gemm(x.float(), xs, w, ws, **ok),
        lambda: ep.expert_gemm(x, xs[:, :1], w, ws, **ok),
        lambda: ep.expert_gemm(x[:, :200], xs, w, ws, **ok),
        lambda: ep.expert_gemm(x, xs, w[:, :, :128].contiguous(), ws, **ok),
        lambda: ep.expert_gemm(x, xs, w, ws[:, :, :1].contiguous(), **ok),
        lambda: ep.expert_gemm(x, xs, w, ws),
        lambda: ep.expert_gemm(x, xs, w, ws, counts=cnt.long(), offsets=off),
        lambda: ep.expert_gemm(x, xs, w, ws, out=torch.empty(8, 255, dtype=torch.bfloat16, device="cuda"), **ok),
        lambda: ep.expert_gemm(x, xs, w, ws, out=torch.empty(8, 256, device="cuda"), **ok),
        lambda: ep.expert_swiglu(x, xs, w[:, :130].contiguous(), ws, **ok),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, ep.EpError)):
            f()
            pytest.fail(f"refusal {i} was accepted")
    # codes off a 16-byte boundary are refused by the library
    flat = torch.zeros(8 * 256 + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ep.EpError):
        ep.expert_gemm(flat[1:1 + 8 * 256].view(8, 256), xs, w, ws, **ok)


def test_packed_descriptors_are_laid_out_like_the_structures():
    """The binding packs the C descriptors as bytes: field for field what the ctypes structures hold."""
    import ctypes
    from combine_get_dispatch_histograms_gb300 import _lib, experts
    for pack, struct_, values in ((experts._ROWS, _lib.EpFp8Rows, (3, 5, 7, 11, 1 << 40)),
                                  (experts._GROUPS, _lib.EpRowGroups, (3, 5, 0, 13, 1 << 35, 9)),
                                  (experts._WEIGHT, _lib.EpFp8Weight, (1 << 41, 5, 7, 11, 13)),
                                  (experts._MOE, _lib.EpMoeWeights, (1 << 41, 5, 0, 1 << 42, 11, 13, 17))):
        raw = pack(*values)
        assert len(raw) == ctypes.sizeof(struct_)
        back = struct_.from_buffer_copy(raw)
        assert tuple(getattr(back, f) or 0 for f, _ in struct_._fields_) == values


@gpu
def test_regions_hold_no_more_than_their_rows():
    cnt, off, hoff, x, xs, w, ws = case([40, 40], 128, 256, seed=81)
    st = ep.new_status()
    counts = torch.tensor([70, 40], dtype=torch.int32, device="cuda")    # regions of 40 rows
    out = ep.expert_gemm(x.view(2, 40, 128), xs.view(2, 40, 1), w, ws, counts=counts, status=st)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(st)
    assert e.value.status == "EP_ERR_CAPACITY"
    for g_ in range(2):
        r = slice(40 * g_, 40 * g_ + 40)
        assert_bf16_close(out[g_], *product64(rows64(x[r], xs[r]), weight64(w[g_], ws[g_])))


@gpu
def test_no_rows_and_no_groups_rows():
    cnt, off, _, x, xs, w, ws = case([3, 4], 128, 128, seed=82)
    assert ep.expert_gemm(x[:0], xs[:0], w, ws, counts=cnt * 0, offsets=off).shape == (0, 128)
    out = torch.full((7, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt * 0, offsets=off, out=out)
    assert (out == 2.0).all()
    codes, scales = ep.expert_swiglu(x[:0], xs[:0], w.view(1, 256, 128), ws.view(1, 2, 1), counts=cnt[:1] * 0, offsets=off[:1])
    assert codes.shape == (0, 128) and scales.shape == (0, 1)


@gpu
def test_offsets_past_32_bits():
    """Rows 60 million elements apart: the last row of x and of the output lies past 2^31 elements and 2^32 bytes."""
    g = gen(83)
    rows, K, N, step = 40, 128, 136, 60_000_000
    q, s = quantize_rows(randn((rows, K), g))
    xb = torch.empty(rows * step, dtype=torch.uint8, device="cuda")
    x = torch.as_strided(xb, (rows, K), (step, 1))
    x.copy_(q)
    ob = torch.empty(rows * step, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(ob, (rows, N), (step, 1))
    w, ws = quantize_weight(randn((1, N, K), g) * K ** -0.5)
    y, err = product64(rows64(q, s), weight64(w[0], ws[0]))
    for expected in (1, 4096):
        out.zero_()
        ep.expert_gemm(x, s, w[0], ws[0], out=out, expected_rows=expected)
        assert_bf16_close(out, y, err)


def test_c_refusals_without_a_gpu():
    from combine_get_dispatch_histograms_gb300 import _lib
    import ctypes
    lib = _lib.load()
    x = _lib.EpFp8Rows(256, 128, 256, 1, 4)
    g = _lib.EpRowGroups(None, None, None, 0, 4, 0)
    w = lambda **k: _lib.EpFp8Weight(*[dict(dict(codes=256, scales=256, groups=1, n=8, k=128), **k)[n] for n in  # noqa: E731
                                       ("codes", "scales", "groups", "n", "k")])
    call = lambda x_, w_: lib.ep_expert_gemm(ctypes.byref(x_), ctypes.byref(g), ctypes.byref(w_), 256, 8, None, None)  # noqa: E731
    assert lib.ep_expert_gemm(None, None, None, None, 0, None, None) == -1
    for bad in (dict(groups=0), dict(groups=5000), dict(n=0), dict(k=100), dict(codes=None), dict(scales=None), dict(codes=257)):
        assert call(x, w(**bad)) == -1, bad
    assert call(_lib.EpFp8Rows(256, 100, 256, 1, 4), w()) == -1        # row stride
    assert call(_lib.EpFp8Rows(256, 128, 256, 0, 4), w()) == -1        # scale stride
    assert call(_lib.EpFp8Rows(256, 128, 256, 1, -1), w()) == -1       # rows
    assert call(_lib.EpFp8Rows(None, 0, None, 0, 0), w()) == 0         # nothing to do
    w13 = w(n=128)
    assert lib.ep_expert_swiglu(ctypes.byref(x), ctypes.byref(g), ctypes.byref(w13), 256, 128, 256, 1, None, None) == -1


@gpu
@pytest.mark.parametrize("form,G,rows,K,N,expected", [("cluster", 3, 140, 1024, 512, 0), ("one", 90, 300, 128, 1024, 64),
                                                      ("pairs", 90, 1000, 128, 1024, 500)])
def test_groups_that_overlap_are_cut_and_flagged(form, G, rows, K, N, expected):
    """Every group claims all rows: more tiles than the rows could have.  Blocks write them beside one another, so that an
    element holds some group's product, or is left alone."""
    from expert_shapes import form_of
    assert form_of(rows, G, N, K, expected) == form
    g = gen(G)
    x, xs = quantize_rows(randn((rows, K), g))
    w, ws = quantize_weight(randn((G, N, K), g) * K ** -0.5)
    cnt, off = torch.full((G,), rows, dtype=torch.int32, device="cuda"), torch.zeros(G, dtype=torch.int32, device="cuda")
    st = ep.new_status()
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, status=st, expected_rows=expected)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(st)
    assert e.value.status == "EP_ERR_CAPACITY"
    ep.expert_swiglu(x, xs, w, ws, counts=cnt, offsets=off, status=st, expected_rows=expected)
    with pytest.raises(ep.EpError):
        ep.check_status(st)
    fits = out == 7.0
    for i in range(G):
        y, err = product64(rows64(x, xs), weight64(w[i], ws[i]))
        fits |= (out.double() - y).abs() <= 2.0 ** -8 * y.abs() + err
    assert fits.all()
    # one group after the other is no overlap
    cnt = torch.tensor([rows] + [0] * (G - 1), dtype=torch.int32, device="cuda")
    ep.expert_gemm(x, xs, w, ws, counts=cnt, offsets=off, out=out, status=st, expected_rows=expected)
    ep.check_status(st)
    assert_bf16_close(out, *product64(rows64(x, xs), weight64(w[0], ws[0])))


def test_tile_walk_stays_within_31_bits():
    """The walk's arithmetic, restated: groups that claim every row, with far more than 2^31 tiles in all, at the most
    tiles that the host lets through; and groups that share none."""
    most_tiles = 1 << 25

    def walk(tiles, most, unit, units):
        """(group, tile of the group) that `unit` takes, and whether tiles were cut off; no sum may pass 31 bits."""
        start = total = 0
        g0, inc, got, t = -32, [], [], unit
        while True:
            at = min(t, most)
            while at >= start + total:
                start += total
                g0 += 32
                if g0 >= len(tiles):
                    return got, False
                inc, run = [], 0
                for v in (tiles[g0:g0 + 32] + [0] * 32)[:32]:
                    run += v
                    inc.append(run)
                total = inc[-1]
                assert start + total < 1 << 31
            if t >= most:
                return got, True
            src = next(i for i in range(32) if at < start + inc[i])
            got.append((g0 + src, at - start - (inc[src - 1] if src else 0)))
            t += units
            assert t < 1 << 31
    huge = [most_tiles] * 4096
    units = 60000                        # a grid has fewer blocks than this
    for unit in (0, 1, units - 1):
        got, cut = walk(huge, most_tiles, unit, units)
        assert cut and got == [(0, t) for t in range(unit, most_tiles, units)]
    parts = [most_tiles // 100 + 3] * 200
    got, cut = walk(parts, most_tiles, 5, units)
    assert cut and [g * parts[0] + r for g, r in got] == list(range(5, most_tiles, units))
    fine = [3, 0, 5, 0] * 100
    seen = sorted(p for unit in range(7) for p in walk(fine, sum(fine), unit, 7)[0])
    assert seen == [(g, r) for g, n in enumerate(fine) for r in range(n)]
    assert not any(walk(fine, sum(fine), unit, 7)[1] for unit in range(7))


@gpu
def test_activation_over_its_range():
    """One code times a scale of any fp32 value: gate and up are exact, all 128 channels of a block are equal, and the
    block's scale is |h| / 448 in fp32.  silu(g) * u is off by at most 8 * 2^-23 of itself, for negative g by |g| * 2^-23
    more; the division rounds to 2^-24.  Below -87 it may be 0."""
    s = torch.cat([torch.logspace(-4, 1.93, 4000, device="cuda"), torch.tensor([85.0, 86.9, 87.5, 89.0, 120.0, 1e4], device="cuda")])
    rows = s.numel()
    x = torch.zeros(rows, 128, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(512, 128, device="cuda")
    w[:128, 0], w[128:256, 0], w[256:, 0] = -1, 1, 1         # gate -s in block 0, s in block 1; up s
    one = torch.ones(4, 1, device="cuda")
    for shape in ("cluster or one", "pairs"):
        G = 1 if shape != "pairs" else 40
        n = rows // G * G
        kw = {} if G == 1 else dict(counts=torch.full((G,), n // G, dtype=torch.int32, device="cuda"),
                                    offsets=torch.arange(0, n, n // G, dtype=torch.int32, device="cuda"), expected_rows=500)
        W, WS = w.to(torch.float8_e4m3fn).expand(G, -1, -1).contiguous(), one.expand(G, -1, -1).contiguous()
        _, scales = ep.expert_swiglu(x[:n].to(torch.float8_e4m3fn), s[:n, None].contiguous(), W, WS, **kw)
        g = torch.stack([-s[:n], s[:n]], 1).double()
        h = (g / (1 + torch.exp(-g)) * s[:n, None].double()).abs()
        d = (scales.double() * 448 - h).abs()
        lim = (8 + g.clamp(max=0).abs() + 1) * 2.0 ** -23 * h + torch.where(g < -87, 88 * 2.0 ** -126 * s[:n, None].double(), 0.0) + 1e-43
        assert (d <= lim).all(), f"{shape}: worst {float((d / lim).max()):.3g} of the bound"


def test_c_refuses_pointers_off_their_elements():
    """A count, an offset or a scale off its 4 bytes would be a misaligned address on the GPU."""
    import ctypes
    from combine_get_dispatch_histograms_gb300 import _lib
    lib = _lib.load()

    def call(fn="gemm", xs=256, ws=256, counts=256, offsets=256, bases=None, out=256, out_scales=256, status=256):
        x = _lib.EpFp8Rows(256, 128, xs, 1, 4)
        g = _lib.EpRowGroups(counts, offsets, bases, 1, 4, 0)
        w = _lib.EpFp8Weight(256, ws, 1, 256, 128)
        p = [ctypes.byref(a) for a in (x, g, w)]
        if fn == "gemm":
            return lib.ep_expert_gemm(*p, out, 256, status, None)
        return lib.ep_expert_swiglu(*p, out, 128, out_scales, 1, status, None)
    for fn in ("gemm", "swiglu"):
        for bad in (dict(xs=258), dict(ws=257), dict(counts=258), dict(offsets=257), dict(bases=258), dict(status=259), dict(out=257)):
            assert call(fn, **bad) == -1, (fn, bad)
            assert b"align" in lib.ep_last_error() or b"output" in lib.ep_last_error()
    assert call("swiglu", out_scales=258) == -1
