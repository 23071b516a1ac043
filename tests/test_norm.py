"""rms_norm and its backward pass against 64 bits.

Bounds, before any run.  A row's sum of squares: at most 8 * 4 terms a thread one after another, then 10 steps of a tree:
relative error 42 * 2^-24; half of it reaches the root, with 2 ulp of rsqrtf, the division by H and eps 25 * 2^-24 + 3 *
2^-24, and two products more: 2^-19 covers n.  dx: the sum of g h has 43 * 2^-24 of the sum of |g h|, so 2^-18 of
|d| + s |g| + s^3 |h| mean |g h| covers it.  dweight: at most 17 rows a block (5000 rows on 304 blocks), 8 warps, 38 + 8
blocks' sums: 71 * 2^-24 of the sum of |terms|, and 2^-19 of each term: 2^-17 covers it.  Then half a step of the output."""
import ctypes

import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import Context, _lib, inputs
from expert_util import gen, randn, rows64

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
SIZES = [(1, 8), (1, 128), (3, 136), (5, 1000), (7, 1024), (9, 1032), (2, 7168), (500, 7168), (5, 8192), (3, 8200), (2, 16384),
         (1000, 512), (5000, 256)]


def make(rows, H, residual, weight, seed):
    g = gen(seed)
    x = randn((rows, H), g).to(BF)
    r = None if residual is None else (3 * randn((rows, H), g)).to(residual)
    return x, r, (1 + 0.2 * randn((H,), g)).to(weight), g


def forward64(h, w, eps):
    h = h.double()
    s = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    return h * s * w.double(), s


def check_y(y, n):
    assert y.dtype == BF and ((y.double() - n).abs() <= (2.0 ** -8 + 2.0 ** -19) * n.abs() + 1e-38).all()


def check_rows(rows, n):
    codes, scales = ep.fp8_row_views(rows, n.shape[-1])
    a = n.abs().reshape(n.shape[0], -1, 128).amax(-1) / 448
    assert ((scales.double() - a).abs() <= 2.0 ** -18 * a).all()
    step = scales.double().repeat_interleave(128, -1)
    d = (rows64(codes, scales) - n).abs()
    assert (d <= (2.0 ** -4 + 2.0 ** -16) * n.abs() + 2.0 ** -10 * step).all()


@gpu
@pytest.mark.parametrize("residual,weight", [(None, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,H", SIZES)
def test_forward(rows, H, residual, weight):
    x, r, w, _ = make(rows, H, residual, weight, rows + H)
    fp8 = H % 128 == 0
    got = ep.rms_norm(x, w, 1e-5, residual=r, fp8=fp8)
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    if r is not None:
        assert torch.equal(got["residual"], h)
    n, _ = forward64(h, w, 1e-5)
    check_y(got["y"], n)
    assert ("rows" in got) == fp8
    if fp8:
        check_rows(got["rows"], n)
        only = ep.rms_norm(x, w, 1e-5, residual=r, y=False, fp8=True)
        assert "y" not in only and torch.equal(only["rows"][:, :H + H // 32], got["rows"][:, :H + H // 32])


def backward64(dy, h, w, dres, eps):
    dy, h, w = dy.double(), h.double(), w.double()
    s = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = dy * w
    dx = s * (g - h * s * s * (g * h).mean(-1, keepdim=True)) + (0 if dres is None else dres.double())
    mag = s * g.abs() + s ** 3 * h.abs() * (g * h).abs().mean(-1, keepdim=True) + (0 if dres is None else dres.double().abs())
    return dx, mag, (dy * h * s).sum(0), (dy * h * s).abs().sum(0)


@gpu
@pytest.mark.parametrize("kind,weight,dres", [(BF, BF, True), (BF, F32, False), (F32, F32, True)])
@pytest.mark.parametrize("rows,H", SIZES)
def test_backward(rows, H, kind, weight, dres):
    h, _, w, g = make(rows, H, None, weight, rows + 2 * H)
    h = (2 * h.float()).to(kind)
    dy = randn((rows, H), g).to(BF)
    d = randn((rows, H), g).to(kind) if dres else None
    dx, dw = ep.rms_norm_backward(dy, h, w, 1e-5, dresidual=d)
    ref, mag, dw64, dwmag = backward64(dy, h, w, d, 1e-5)
    assert dx.dtype == kind and dw.dtype == F32
    assert ((dx.double() - ref).abs() <= HALF[kind] * ref.abs() + 2.0 ** -18 * mag).all()
    assert ((dw.double() - dw64).abs() <= 2.0 ** -17 * dwmag).all()
    again = ep.rms_norm_backward(dy, h, w, 1e-5, dresidual=d)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@gpu
def test_backward_against_differences():
    """dx and dweight along a direction, against the 64-bit forward's central difference (its third-order term: 1e-8 here)."""
    rows, H, eps = 6, 264, 1e-5
    h, _, w, g = make(rows, H, None, F32, 3)
    h, dy = h.float(), randn((rows, H), g).to(BF)
    dx, dw = ep.rms_norm_backward(dy, h, w, eps)
    u, v, t = randn((rows, H), g).double(), randn((H,), g).double(), 1e-4
    f = lambda k: (dy.double() * forward64(h.double() + k * u, w.double() + k * v, eps)[0]).sum()  # noqa: E731
    numeric = (f(t) - f(-t)) / (2 * t)
    exact = (dx.double() * u).sum() + (dw.double() * v).sum()
    scale = (dx.double() * u).abs().sum() + (dw.double() * v).abs().sum()
    assert abs(numeric - exact) <= 1e-5 * scale


@gpu
def test_strides_three_dimensions_and_in_place():
    R, T, H = 3, 5, 256
    g = gen(4)
    wide = randn((R, T, 2 * H), g).to(BF)
    x, w = wide[..., H:], torch.ones(H, device="cuda")
    r = randn((R, T, H), g)
    ref = ep.rms_norm(x.contiguous(), w, residual=r)
    h, y = ref["residual"], ref["y"]
    outer = torch.full((R, T, 3 * H), 7.0, device="cuda", dtype=BF)
    got = ep.rms_norm(x, w, residual=r, out={"residual": r, "y": outer[..., H:2 * H]})
    assert got["residual"] is r and torch.equal(r, h) and torch.equal(outer[..., H:2 * H], y)
    assert (outer[..., :H] == 7).all() and (outer[..., 2 * H:] == 7).all()
    z = x.contiguous()
    assert torch.equal(ep.rms_norm(z, w, out={"y": z})["y"], ep.rms_norm(x.contiguous(), w)["y"])
    dy, d = randn((R, T, H), g).to(BF), randn((R, T, H), g)
    dx, dw = ep.rms_norm_backward(dy, h, w, dresidual=d)
    dx2, dw2 = ep.rms_norm_backward(dy, h, w, dresidual=d, out=(d, torch.full((H,), 9.0, device="cuda")))
    assert dx2 is d and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    assert ep.rms_norm(x[0, 0], w)["y"].shape == (H,)


@gpu
def test_rows_further_apart_than_32_bits_reach():
    H, far = 1032, (1 << 30) + 8
    big = torch.empty(3 * far, dtype=BF, device="cuda")
    x = torch.as_strided(big, (3, H), (far, 1))
    x.copy_(randn((3, H), gen(12)))
    w = torch.ones(H, device="cuda")
    c = x.clone()
    assert torch.equal(ep.rms_norm(x, w)["y"], ep.rms_norm(c, w)["y"])
    for a, b in zip(ep.rms_norm_backward(x, x, w, dresidual=x), ep.rms_norm_backward(c, c, w, dresidual=c)):
        assert torch.equal(a, b)
    ep.rms_norm(x, w, out={"y": x})
    assert torch.equal(x, ep.rms_norm(c, w)["y"])


@gpu
def test_no_rows():
    w, x = torch.ones(128, device="cuda"), torch.empty(0, 128, device="cuda", dtype=BF)
    got = ep.rms_norm(x, w, residual=x, fp8=True)
    assert got["y"].shape == (0, 128) and got["rows"].shape[0] == 0
    dx, dw = ep.rms_norm_backward(x, x, w, out=(x, torch.full((128,), 5.0, device="cuda")))
    assert (dw == 0).all()


@gpu
@pytest.mark.parametrize("rows,H", [(300, 256), (500, 2048), (3, 16384)])
def test_given_workspaces(rows, H):
    x, _, w, g = make(rows, H, None, BF, 14)
    dy = randn((rows, H), g).to(BF)
    want = ep.rms_norm_backward(dy, x, w)
    ws = torch.full((ep.rms_norm_backward_workspace(rows, H),), 255, dtype=torch.uint8, device="cuda")   # NaN, if it were read
    for _ in range(2):
        got = ep.rms_norm_backward(dy, x, w, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ep.EpError):
        ep.rms_norm_backward(dy, x, w, workspace=ws[:-16])
    with pytest.raises(ValueError):
        ep.rms_norm_backward(dy, x, w, workspace=ws[::2])


@gpu
def test_zeros_nan_and_infinity_stay_in_their_rows():
    rows, H = 5, 384
    x, _, w, _ = make(rows, H, None, F32, 8)
    x[0] = 0
    x[2, 17] = float("nan")
    x[4, 5] = float("inf")
    got = ep.rms_norm(x, w, fp8=True)
    codes, scales = ep.fp8_row_views(got["rows"], H)
    assert (got["y"][0] == 0).all() and (scales[0] == 0).all()
    assert torch.isnan(got["y"][2]).all() and torch.isnan(scales[2]).all()
    assert torch.isnan(got["y"][4, 5])                       # inf * 0
    good = [1, 3]
    check_y(got["y"][good], forward64(x, w, 1e-6)[0][good])
    dx, _ = ep.rms_norm_backward(x.clone().fill_(1), x, w)
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[[0, 1, 3]]).all()


@gpu
def test_rows_are_what_dispatch_carries():
    """A context's FP8 dispatch of the norm's rows equals the norm's rows at the places of the permuted layout."""
    R, E, K, T, H = 2, 8, 2, 20, 256
    x = inputs.random_x(R, T, H, 1).cuda()
    idx, v = inputs.random_topk(R, E, K, T, 3).cuda(), inputs.random_weights(R, T, K, 2).cuda()
    rows = ep.rms_norm(x, torch.ones(H, device="cuda"), fp8=True)["rows"]
    ctx = Context(R, E, K, T, H)
    assert rows.shape == (R * T, ctx.fp8_row_bytes)
    h = ctx.notify_dispatch(idx, ctx.get_dispatch_layout(idx))
    got = ctx.dispatch_permuted_fp8(rows, idx, v, h)
    ctx.check()
    assert torch.equal(got["permuted_xq"][:, :H + H // 32], rows[got["perm_src_token"].long()][:, :H + H // 32])


@gpu
def test_on_a_stream_and_in_a_graph():
    rows, H = 64, 1024
    x, r, w, g = make(rows, H, BF, BF, 11)
    dy = randn((rows, H), g).to(BF)
    want = ep.rms_norm(x, w, residual=r)
    want_b = ep.rms_norm_backward(dy, want["residual"], w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ep.rms_norm(x, w, residual=r, stream=side)
    got_b = ep.rms_norm_backward(dy, got["residual"], w, stream=side)
    side.synchronize()
    assert torch.equal(got["y"], want["y"]) and torch.equal(got_b[1], want_b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ep.rms_norm(x, w, residual=r)
        got_b = ep.rms_norm_backward(dy, got["residual"], w)
    x.copy_(randn((rows, H), g).to(BF))
    for _ in range(2):
        graph.replay()
    want = ep.rms_norm(x, w, residual=r)
    want_b = ep.rms_norm_backward(dy, want["residual"], w)
    assert torch.equal(got["y"], want["y"]) and torch.equal(got_b[0], want_b[0]) and torch.equal(got_b[1], want_b[1])


def test_refusals_of_the_binding():
    x, w = torch.zeros(4, 128, dtype=BF), torch.ones(128)
    with pytest.raises(ValueError, match="CUDA device"):
        ep.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA device"):
        ep.rms_norm_backward(x, x, w)


@gpu
def test_refusals_on_the_gpu():
    x, w = torch.zeros(4, 136, dtype=BF, device="cuda"), torch.ones(136, device="cuda")
    for call in (lambda: ep.rms_norm(x.float(), w), lambda: ep.rms_norm(x, w[:128]), lambda: ep.rms_norm(x, w, fp8=True),
                 lambda: ep.rms_norm(x, w, residual=x[:3]), lambda: ep.rms_norm(x, w, residual=x.half()),
                 lambda: ep.rms_norm(x, w.half()), lambda: ep.rms_norm(x, w, out={"residual": x}),
                 lambda: ep.rms_norm(x[:, ::2], w[:68]), lambda: ep.rms_norm_backward(x, x, w, dresidual=x.float()),
                 lambda: ep.rms_norm(x, w, out={"y": x[:2]}), lambda: ep.rms_norm(x.view(-1)[::4], w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ep.rms_norm(x[:, 1:129], w[:128]), lambda: ep.rms_norm(x, w, eps=0.0),
                 lambda: ep.rms_norm(x[:, :132], w[:132].contiguous()), lambda: ep.rms_norm(x, w, y=False),
                 lambda: ep.rms_norm_backward(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: ep.rms_norm(torch.zeros(1, 16392, dtype=BF, device="cuda"), torch.ones(16392, device="cuda"))):
        with pytest.raises(ep.EpError):
            call()


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(hidden=0), dict(hidden=12), dict(hidden=16392), dict(eps=0.0), dict(eps=float("nan")), dict(rtype=2), dict(wtype=-1),
    dict(weight=None), dict(x=None), dict(x=0x1008), dict(xs=120), dict(xs=129), dict(y=None), dict(residual=0x2000), dict(res_out=0x2000),
    dict(fp8=0x3000, fs=128), dict(fp8=0x3008, fs=144), dict(hidden=136, xs=136, ys=136, fp8=0x3000, fs=160)])
def test_refusals_of_the_library(change):
    """Addresses that are never read: every call is refused on the host."""
    a = dict(x=0x1000, xs=128, residual=None, rs=128, rtype=0, weight=0x4000, wtype=1, eps=1e-6, rows=4, hidden=128, res_out=None, y=0x5000,
             ys=128, fp8=None, fs=0) | change
    rc = _lib.load().ep_rms_norm(a["x"], a["xs"], a["residual"], a["rs"], a["rtype"], a["weight"], a["wtype"], a["eps"], a["rows"],
                                 a["hidden"], a["res_out"], 128, a["y"], a["ys"], a["fp8"], a["fs"], None)
    assert rc == -1 and _lib.load().ep_last_error().startswith(b"ep_rms_norm:")


@pytest.mark.parametrize("change", [dict(dweight=None), dict(dweight=0x6002), dict(dy=None), dict(h=0x1004), dict(dx=None), dict(dres=0x1001),
                                    dict(dys=64), dict(hidden=20), dict(rows=1 << 31)])
def test_refusals_of_the_library_backward(change):
    a = dict(dy=0x1000, dys=128, h=0x2000, dres=None, rows=4, hidden=128, dx=0x3000, dweight=0x6000) | change
    rc = _lib.load().ep_rms_norm_backward(a["dy"], a["dys"], a["h"], 128, 0, 0x4000, 1, 1e-6, a["dres"], 128, a["rows"], a["hidden"],
                                          a["dx"], 128, a["dweight"], 0x7000, 1 << 30, None)
    assert rc == -1 and _lib.load().ep_last_error().startswith(b"ep_rms_norm_backward:")
