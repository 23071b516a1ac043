"""MXFP4 rows and products against 64 bits.

Bounds, before any run.  Quantisation is exact: every code and scale equals the definition's.  A product's sum: K / 64
instructions, each at most two roundings or truncations at 2^-23 of what S = sum |x||w| bounds, and 8 to spare:
(K / 64 + 8) 2^-22 S; then half a step of bf16.  A requantised h lies between the codes of h - err and h + err, err as the FP8
products' with that sum."""
import ctypes

import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import Context, _lib, fp4, inputs
from combine_get_dispatch_histograms_gb300.fp4 import fp4_row_views
from expert_util import assert_bf16_close, gen, randn, silu64
from test_experts import LONG, RAGGED, groups_of

gpu = pytest.mark.gpu
BF = torch.bfloat16
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def round4(a):
    """The nearest e2m1 value of a in 64 bits, ties to the even code, saturated."""
    m, q = a.abs(), torch.zeros_like(a)
    for i, edge in enumerate([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]):
        q = torch.where(m >= edge if i % 2 else m > edge, GRID[i + 1], q)
    return torch.copysign(q, a)


def scale_byte(amax):
    """b of a block's largest magnitude in 64 bits; 255 where it is not finite."""
    e = torch.frexp(amax).exponent.long() - 1 - 2 + 127
    b = torch.where(amax > 0, e, 0).clamp(0, 254)
    return torch.where(torch.isfinite(amax), b, 255)


def values4(codes, scales):
    t = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=codes.device)
    t[8] = -0.0
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).flatten(-2)
    s = torch.where(scales == 255, float("nan"), power(scales.long() - 127))
    return v * s.repeat_interleave(32, -1)


def quantize_ref(x):
    """(codes, scales) of finite rows in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    s = scale_byte(b.abs().amax(-1))
    q = round4(b / power(s - 127)[..., None]).flatten(-2)
    code = torch.zeros_like(q, dtype=torch.uint8)
    for i, v in enumerate(GRID):
        code = torch.where(q.abs() == v, i, code)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.to(torch.uint8)


def product64(x, w):
    return x @ w.t(), (x.shape[1] // 64 + 8) * 2.0 ** -22 * (x.abs() @ w.abs().t())


def swiglu64(x, w13):
    n = w13.shape[0] // 2
    y, e = product64(x, w13)
    g, u = y[:, :n], y[:, n:]
    h = silu64(g) * u
    return h, 1.1 * e[:, :n] * u.abs() + silu64(g).abs() * e[:, n:] + 1.1 * e[:, :n] * e[:, n:] + 2.0 ** -20 * h.abs()


def assert_fp4_close(codes, scales, h, err):
    a, e = (t.reshape(h.shape[0], -1, 32) for t in (h.abs(), err))
    lo, hi = scale_byte((a - e).clamp(min=0).amax(-1)), scale_byte((a + e).amax(-1))
    b = scales.long()
    assert ((b >= lo) & (b <= hi)).all(), "scales"
    unit = power(b - 127).repeat_interleave(32, -1)
    got = values4(codes, torch.full_like(scales, 127))
    assert (got >= round4((h - err) / unit)).all() and (got <= round4((h + err) / unit)).all(), "codes"


def rows4(rows, K, g):
    return quantize_ref(randn((rows, K), g))


def weight4(G, N, K, g):
    c, s = quantize_ref((randn((G, N, K), g) * K ** -0.5).view(-1, K))
    return c.view(G, N, K // 2), s.view(G, N, K // 32)


@gpu
@pytest.mark.parametrize("rows,K", [(1, 128), (3, 384), (777, 1408), (4096, 7168), (5, 16384)])
def test_quantize(rows, K):
    g = gen(rows + K)
    x = (randn((rows, K), g) * torch.exp2(torch.randint(-140, 120, (rows, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)).to(BF)
    x = torch.where(torch.isfinite(x), x, 0).to(BF)
    x[0, :32] = 0
    codes, scales = ep.quantize_fp4(x)
    want = quantize_ref(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@gpu
def test_quantize_every_bf16_value():
    """Each bf16 value beside each of four block maxima; ties and saturation among them."""
    v = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(BF)
    v = v[torch.isfinite(v)]
    v = torch.cat([v, v.new_zeros(-len(v) % 62)]).view(-1, 31 * 2)
    for top in (2.0 ** 127, 1.9921875, 2.0 ** -126, 2.0 ** -133):
        t = torch.full_like(v[:, :1], top)
        x = torch.where(torch.cat([t, v[:, :31], t, v[:, 31:]], 1).abs() <= top, torch.cat([t, v[:, :31], t, v[:, 31:]], 1), t)
        x = torch.cat([x, x], 1)                                # 128 channels
        codes, scales = ep.quantize_fp4(x)
        want = quantize_ref(x)
        assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])


@gpu
def test_quantize_keeps_nan_and_infinity_in_their_blocks():
    x = randn((4, 256), gen(1)).to(BF)
    x[1, 40], x[2, 255], x[3, 0] = float("nan"), float("inf"), -float("inf")
    codes, scales = ep.quantize_fp4(x)
    bad = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 7] = bad[3, 0] = True
    assert torch.equal(scales == 255, bad)
    ok = torch.nan_to_num(x.float(), 0, 0, 0).to(BF)
    want = quantize_ref(ok)
    keep = ~bad.repeat_interleave(16, 1)
    assert torch.equal(codes[keep], want[0][keep])


@gpu
def test_quantize_strides_regions_and_rows():
    g = gen(2)
    wide = randn((3, 10, 512), g).to(BF)
    x = wide[..., 128:384]
    want = quantize_ref(x.reshape(-1, 256))
    codes, scales = ep.quantize_fp4(x)
    assert torch.equal(codes.view(-1, 128), want[0]) and torch.equal(scales.view(-1, 8), want[1])
    rows = torch.full((30, 160), 9, dtype=torch.uint8, device="cuda")
    ep.quantize_fp4(x.reshape(-1, 256), out=fp4_row_views(rows, 256))
    assert torch.equal(rows[:, :128], want[0]) and torch.equal(rows[:, 128:136], want[1]) and (rows[:, 136:] == 9).all()
    assert ep.quantize_fp4(x[0, :0])[0].shape == (0, 128)


@gpu
@pytest.mark.parametrize("K,N", [(128, 16), (256, 64), (1024, 192)])
def test_gemm_of_one_block_exactly(K, N):
    """Small whole numbers, scales of one: every sum is exact, so a misplaced code, scale or row shows."""
    g = gen(K + N)
    rows = 128
    x = torch.randint(0, 3, (rows, K), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float()
    xs = torch.randint(-3, 4, (rows, K // 32), generator=g, device="cuda")
    ws = torch.randint(-3, 4, (N, K // 32), generator=g, device="cuda")

    def codes_of(v):
        c = torch.zeros_like(v, dtype=torch.uint8)
        for i, m in enumerate(GRID):
            c = torch.where(v.abs() == m, i, c)
        c = c | ((v < 0).to(torch.uint8) << 3)
        return c[:, 0::2] | (c[:, 1::2] << 4)
    xc, wc = codes_of(x), codes_of(w)
    xb, wb = (xs + 127).to(torch.uint8), (ws + 127).to(torch.uint8)
    y = values4(xc, xb) @ values4(wc, wb).t()
    got = ep.expert_gemm_fp4(xc, xb, wc, wb)
    assert torch.equal(got, y.to(BF))


@gpu
@pytest.mark.parametrize("K,N", [(128, 128), (128, 1), (256, 130), (640, 256), (1408, 600), (2048, 1099), (512, 8), (384, 257), (768, 193)])
@pytest.mark.parametrize("counts", [[1], [5, 0, 64], RAGGED, LONG])
def test_gemm_ragged(K, N, counts):
    cnt, off, hoff, rows = groups_of(counts, 3)
    g = gen(K + N)
    x, xs = rows4(rows, K, g)
    w, ws = weight4(len(counts), N, K, g)
    st = ep.new_status()
    out = torch.full((rows, N), 7.0, dtype=BF, device="cuda")
    ep.expert_gemm_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=out, status=st)
    ep.check_status(st)
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(hoff, counts)):
        own[o:o + c] = True
        if c:
            y, err = product64(values4(x[o:o + c], xs[o:o + c]), values4(w[e], ws[e]))
            assert_bf16_close(out[o:o + c], y, err, f"group {e}")
    assert (out[~own] == 7.0).all(), "rows of no group were written"


@gpu
@pytest.mark.parametrize("K,I", [(128, 128), (640, 384), (1024, 256), (4096, 128), (2048, 640)])
@pytest.mark.parametrize("counts", [[1], [5, 0, 64], RAGGED, LONG])
def test_swiglu_ragged(K, I, counts):
    cnt, off, hoff, rows = groups_of(counts, 2)
    g = gen(K + I)
    x, xs = rows4(rows, K, g)
    w, ws = weight4(len(counts), 2 * I, K, g)
    st = ep.new_status()
    codes = torch.full((rows, I // 2), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, I // 32), 5, dtype=torch.uint8, device="cuda")
    ep.expert_swiglu_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=(codes, scales), status=st)
    ep.check_status(st)
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(hoff, counts)):
        own[o:o + c] = True
        if c:
            assert_fp4_close(codes[o:o + c], scales[o:o + c], *swiglu64(values4(x[o:o + c], xs[o:o + c]), values4(w[e], ws[e])))
    assert (codes[~own] == 9).all() and (scales[~own] == 5).all(), "rows of no group were written"


@gpu
@pytest.mark.parametrize("rows", [1, 2, 33, 127, 128, 129, 256, 500])
@pytest.mark.parametrize("K,N", [(2048, 512), (128, 77), (7168, 256), (4096, 4096), (1280, 9728)])
def test_dense(rows, K, N):
    g = gen(rows + K)
    x, xs = rows4(rows, K, g)
    w, ws = weight4(1, N, K, g)
    assert_bf16_close(ep.expert_gemm_fp4(x, xs, w[0], ws[0]), *product64(values4(x, xs), values4(w[0], ws[0])))
    if N % 256 == 0:
        codes, scales = ep.expert_swiglu_fp4(x, xs, w[0], ws[0])
        assert_fp4_close(codes, scales, *swiglu64(values4(x, xs), values4(w[0], ws[0])))


@gpu
@pytest.mark.parametrize("expected", [1, 100000])
@pytest.mark.parametrize("K,N", [(128, 256), (640, 512), (1408, 768), (2048, 1280), (7168, 256)])
def test_both_shapes_on_long_and_ragged_groups(K, N, expected):
    """One block a tile or two, whatever the groups hold."""
    for counts in (LONG, RAGGED):
        cnt, off, hoff, rows = groups_of(counts, 2)
        g = gen(K + N + expected)
        x, xs = rows4(rows, K, g)
        w, ws = weight4(len(counts), N, K, g)
        out = torch.full((rows, N), 7.0, dtype=BF, device="cuda")
        ep.expert_gemm_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=out, expected_rows=expected)
        hc, hs = (torch.full((rows, n), 7, dtype=torch.uint8, device="cuda") for n in (N // 4, N // 64))
        ep.expert_swiglu_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=(hc, hs), expected_rows=expected)
        own = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for e, (o, c) in enumerate(zip(hoff, counts)):
            own[o:o + c] = True
            if c:
                X, W = values4(x[o:o + c], xs[o:o + c]), values4(w[e], ws[e])
                assert_bf16_close(out[o:o + c], *product64(X, W), f"group {e}")
                assert_fp4_close(hc[o:o + c], hs[o:o + c], *swiglu64(X, W))
        assert (out[~own] == 7.0).all() and (hc[~own] == 7).all() and (hs[~own] == 7).all()


@gpu
@pytest.mark.parametrize("K,N", [(640, 224), (1408, 512), (640, 896), (384, 1099), (1152, 1280), (640, 2304), (256, 4099), (2304, 2048)])
def test_every_tile_width_gives_the_same(K, N):
    """The rows that a caller expects choose the tiles' width, not what comes out: K is summed in the same order by each."""
    for counts in (RAGGED, LONG, [0, 700, 1, 130, 2]):
        cnt, off, hoff, rows = groups_of(counts, 2)
        g = gen(K + N)
        x, xs = rows4(rows, K, g)
        w, ws = weight4(len(counts), N, K, g)
        st = ep.new_status()
        first = None
        for expected in (1, 200, 300, 600, 1000, 4000, 2 ** 40):
            out = torch.full((rows, N + 5), 7.0, dtype=BF, device="cuda")[:, :N]  # rows not on 16 bytes
            wide = torch.full((rows, (N + 7) // 8 * 8), 7.0, dtype=BF, device="cuda")[:, :N]
            got = [ep.expert_gemm_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=o, status=st, expected_rows=expected) for o in (out, wide)]
            if N % 256 == 0:
                h = tuple(torch.full((rows, n), 7, dtype=torch.uint8, device="cuda") for n in (N // 4, N // 64))
                got += ep.expert_swiglu_fp4(x, xs, w, ws, counts=cnt, offsets=off, out=h, status=st, expected_rows=expected)
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got)) and torch.equal(out, wide)
            for o in (out, wide):
                base = torch.as_strided(o, (rows, o.stride(0)), (o.stride(0), 1))
                assert (base[:, N:] == 7).all(), "written past the rows' ends"
        ep.check_status(st)
        own = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for e, (o, c) in enumerate(zip(hoff, counts)):
            own[o:o + c] = True
            if c:
                X, W = values4(x[o:o + c], xs[o:o + c]), values4(w[e], ws[e])
                assert_bf16_close(first[0][o:o + c], *product64(X, W), f"group {e}")
                if N % 256 == 0:
                    assert_fp4_close(first[2][o:o + c], first[3][o:o + c], *swiglu64(X, W))
        assert all((t[~own] == 7).all() for t in first), "rows of no group were written"


@gpu
def test_regions_with_and_without_counts():
    E, cap, K, N = 5, 40, 384, 200
    g = gen(5)
    x, xs = rows4(E * cap, K, g)
    x, xs = x.view(E, cap, -1), xs.view(E, cap, -1)
    w, ws = weight4(E, N, K, g)
    cnt = torch.tensor([0, 40, 3, 17, 1], dtype=torch.int32, device="cuda")
    out = torch.full((E, cap, N), 7.0, dtype=BF, device="cuda")
    ep.expert_gemm_fp4(x, xs, w, ws, counts=cnt, out=out)
    full = ep.expert_gemm_fp4(x, xs, w, ws)
    for e, c in enumerate(cnt.tolist()):
        y, err = product64(values4(x[e], xs[e]), values4(w[e], ws[e]))
        assert_bf16_close(full[e], y, err)
        assert torch.equal(out[e, :c], full[e, :c]) and (out[e, c:] == 7).all()


@gpu
def test_rows_outside_the_arrays_are_cut_off_and_flagged():
    K, N = 256, 100
    g = gen(6)
    x, xs = rows4(50, K, g)
    w, ws = weight4(2, N, K, g)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st = ep.new_status()
    out = torch.full((50, N), 7.0, dtype=BF, device="cuda")
    ep.expert_gemm_fp4(x, xs, w, ws, counts=i32(10, 1000), offsets=i32(0, 40), out=out, status=st)
    with pytest.raises(ep.EpError) as e:
        ep.check_status(st)
    assert e.value.code == -3
    assert_bf16_close(out[40:], *product64(values4(x[40:], xs[40:]), values4(w[1], ws[1])))
    assert (out[10:40] == 7).all()


@gpu
def test_rows_further_apart_than_32_bits_reach():
    K, N, far = 256, 100, (1 << 30) + 16
    g = gen(13)
    x = torch.as_strided(torch.empty(3 * far, dtype=BF, device="cuda"), (3, K), (far, 1))
    x.copy_(randn((3, K), g))
    big = torch.empty(6 * far, dtype=torch.uint8, device="cuda")
    codes, scales = torch.as_strided(big, (3, K // 2), (2 * far, 1)), torch.as_strided(big, (3, K // 32), (2 * far, 1), 1024)
    ep.quantize_fp4(x, out=(codes, scales))
    want = ep.quantize_fp4(x.contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    w, ws = weight4(1, N, K, g)
    out = torch.as_strided(torch.empty(3 * far, dtype=BF, device="cuda"), (3, N), (far, 1))
    ep.expert_gemm_fp4(codes, scales, w[0], ws[0], out=out)
    assert torch.equal(out, ep.expert_gemm_fp4(*want, w[0], ws[0]))


@gpu
def test_a_nan_stays_in_its_row_and_column():
    K, N, rows = 512, 256, 130
    g = gen(7)
    x, xs = rows4(rows, K, g)
    w, ws = weight4(1, N, K, g)
    xs[129, 3] = 255
    ws[0, 200, 15] = 255
    y = ep.expert_gemm_fp4(x, xs, w[0], ws[0])
    bad = torch.zeros(rows, N, dtype=torch.bool, device="cuda")
    bad[129] = True
    bad[:, 200] = True
    assert torch.equal(torch.isnan(y), bad)
    ws[0, 200, 15] = 120
    codes, scales = ep.expert_swiglu_fp4(x, xs, w[0], ws[0])
    assert (scales[129] == 255).all() and (scales[:129] < 255).all()


@gpu
def test_layouts_of_rows_and_outputs():
    """FP4 rows with their scales behind the codes, odd row strides of scales, outputs in wider and unaligned arrays."""
    rows, K, N = 70, 640, 120
    g = gen(8)
    x, xs = rows4(rows, K, g)
    w, ws = weight4(1, N, K, g)
    want = ep.expert_gemm_fp4(x, xs, w[0], ws[0])
    both = torch.zeros(rows, (K // 2 + K // 32 + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    c, s = fp4_row_views(both, K)
    c.copy_(x), s.copy_(xs)
    assert torch.equal(ep.expert_gemm_fp4(c, s, w[0], ws[0]), want)
    odd = torch.zeros(rows, K // 32 + 4, dtype=torch.uint8, device="cuda")
    odd[:, 4:] = xs
    assert torch.equal(ep.expert_gemm_fp4(x, odd[:, 4:], w[0], ws[0]), want)
    for lead, width in ((0, 128), (8, 136), (1, 131), (16, 160)):
        out = torch.full((rows, width), 7.0, dtype=BF, device="cuda")
        ep.expert_gemm_fp4(x, xs, w[0], ws[0], out=out[:, lead:lead + N])
        assert torch.equal(out[:, lead:lead + N], want) and (out[:, :lead] == 7).all() and (out[:, lead + N:] == 7).all()


@gpu
@pytest.mark.parametrize("R,E,K,T,H,I,align", [(4, 8, 2, 40, 128, 128, 1), (2, 16, 4, 300, 512, 384, 1), (4, 12, 3, 65, 256, 640, 16)])
def test_experts_over_a_dispatch(R, E, K, T, H, I, align):
    x, v = inputs.random_x(R, T, H, 1).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    idx = inputs.random_topk(R, E, K, T, 3, mask_p=0.1).cuda()
    g = gen(9)
    w13, s13 = weight4(E, 2 * I, H, g)
    w2, s2 = weight4(E, H, I, g)
    ctx = Context(R, E, K, T, H, expert_alignment=align)
    rows = ctx.quantize_fp4(x)
    assert rows.shape == (R * T, ctx.fp4_row_bytes)
    _, h = ctx.layout_notify(idx, wait=False)
    perm = ctx.dispatch_permuted_fp4(rows, idx, v, h)
    hid = ctx.expert_swiglu_fp4(h, perm["permuted_xq"], w13, s13)
    y = ctx.expert_gemm_fp4(h, hid, w2, s2)
    out = ctx.combine(h, y, idx, v)
    ctx.check()
    codes, scales = quantize_ref(x.view(-1, H))
    X, J, V = values4(codes, scales), idx.view(-1, K), v.view(-1, K).double()
    ref = torch.zeros(R * T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(J == e, as_tuple=True)
        hh, _ = swiglu64(X[t], values4(w13[e], s13[e]))
        ref.index_add_(0, t, V[t, k][:, None] * (values4(*quantize_ref(hh)) @ values4(w2[e], s2[e]).t()).to(BF).double())
    # bf16 of y and of the sum: 2^-9 / sqrt(3) each in the mean square; a code of h rounds the other way once in 10^4 at most,
    # a quarter of itself: 2.5e-3
    assert float((out.view(-1, H).double() - ref).norm() / ref.norm()) < 5e-3


@gpu
def test_streams_and_graphs():
    rows, K, I = 200, 512, 256
    g = gen(10)
    x = randn((rows, K), g).to(BF)
    w13, s13 = weight4(1, 2 * I, K, g)
    w2, s2 = weight4(1, K, I, g)

    def step(stream=None):
        c, s = ep.quantize_fp4(x, stream=stream)
        h, hs = ep.expert_swiglu_fp4(c, s, w13[0], s13[0], stream=stream)
        return ep.expert_gemm_fp4(h, hs, w2[0], s2[0], stream=stream)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(randn((rows, K), g))
    for _ in range(3):
        graph.replay()
    assert torch.equal(got, step())


def test_refusals_of_the_binding():
    x = torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: ep.quantize_fp4(torch.zeros(4, 128, dtype=BF)), lambda: ep.expert_gemm_fp4(x, x, x, x),
                 lambda: ep.expert_swiglu_fp4(x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@gpu
def test_refusals_on_the_gpu():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x, xs, w, ws = u8(4, 64), u8(4, 4), u8(256, 64), u8(256, 4)
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: ep.quantize_fp4(torch.zeros(4, 96, dtype=BF, device="cuda")), lambda: ep.quantize_fp4(torch.zeros(4, 128, device="cuda")),
                 lambda: ep.expert_gemm_fp4(x[:, :32], xs, w, ws), lambda: ep.expert_gemm_fp4(x, xs[:, :2], w, ws),
                 lambda: ep.expert_gemm_fp4(x, xs, w[:, :32], ws), lambda: ep.expert_gemm_fp4(x, xs, w, ws[:128]),
                 lambda: ep.expert_gemm_fp4(x, xs, w.view(2, 128, 64), ws.view(2, 128, 4)),
                 lambda: ep.expert_gemm_fp4(x, xs, w, ws, counts=i32), lambda: ep.expert_gemm_fp4(x.view(2, 2, 64), xs.view(2, 2, 4), w, ws),
                 lambda: ep.expert_gemm_fp4(x, xs, w, ws, out=torch.zeros(4, 255, dtype=BF, device="cuda")),
                 lambda: ep.expert_swiglu_fp4(x, xs, w[:128], ws[:128]), lambda: ep.expert_gemm_fp4(x.float(), xs, w, ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ep.EpError):
        ep.expert_gemm_fp4(u8(4, 72)[:, 8:], xs, w, ws)             # rows 72 bytes apart


def _descriptors(x=0x1000, xstride=64, xscales=0x2000, sstride=4, rows=4, w=0x4000, wscales=0x5000, groups=1, n=256, k=128, counts=0, per=0):
    return fp4._ROWS(x, xstride, xscales, sstride, rows), fp4._GROUPS(counts, 0, 0, per, rows, 0), fp4._WEIGHT(w, wscales, groups, n, k)


@pytest.mark.parametrize("change", [dict(groups=0), dict(groups=4097), dict(n=0), dict(k=64), dict(k=192), dict(w=0), dict(w=0x4008), dict(wscales=0x5002),
                                    dict(rows=-1), dict(x=0), dict(x=0x1004), dict(xscales=0x2001), dict(xstride=48), dict(xstride=72),
                                    dict(sstride=2), dict(sstride=6), dict(counts=2)])
def test_refusals_of_the_library(change):
    """Addresses that are never read: every call is refused on the host."""
    lib = _lib.load()
    d = _descriptors(**change)
    assert len(d[0]) == ctypes.sizeof(_lib.EpFp8Rows) and len(d[2]) == ctypes.sizeof(_lib.EpFp8Weight)
    assert lib.ep_expert_gemm_fp4(*d, 0x8000, 256, None, None) == -1 and lib.ep_last_error().startswith(b"ep_expert_gemm_fp4:")
    assert lib.ep_expert_swiglu_fp4(*d, 0x8000, 64, 0x9000, 4, None, None) == -1


def test_refused_outputs_and_quantisation():
    lib = _lib.load()
    d = _descriptors()
    assert lib.ep_expert_gemm_fp4(*d, None, 256, None, None) == -1
    assert lib.ep_expert_gemm_fp4(*d, 0x8001, 256, None, None) == -1
    assert lib.ep_expert_gemm_fp4(*d, 0x8000, 255, None, None) == -1
    assert lib.ep_expert_gemm_fp4(*d, 0x8000, 256, 0x3, None) == -1
    for out, stride, scales, sstride in ((None, 64, 0x9000, 4), (0x8008, 64, 0x9000, 4), (0x8000, 48, 0x9000, 4), (0x8000, 72, 0x9000, 4),
                                         (0x8000, 64, None, 4), (0x8000, 64, 0x9001, 4), (0x8000, 64, 0x9000, 2)):
        assert lib.ep_expert_swiglu_fp4(*d, out, stride, scales, sstride, None, None) == -1
    assert lib.ep_expert_swiglu_fp4(*_descriptors(n=384), 0x8000, 96, 0x9000, 8, None, None) == -1
    good = [0x1000, 128, 4, 128, 0x2000, 64, 0x3000, 4]
    for i, v in ((0, None), (0, 0x1008), (1, 120), (1, 132), (2, -1), (3, 64), (3, 0), (4, None), (4, 0x2004), (5, 56), (5, 48), (6, 0x3001), (7, 2)):
        assert lib.ep_quantize_fp4(*(good[:i] + [v] + good[i + 1:]), None) == -1
    assert lib.ep_fp4_row_bytes(7168) == 3808 and lib.ep_fp4_row_bytes(128) == 80 and lib.ep_fp4_row_bytes(0) == 0
