"""rms_norm and its backward pass where every block or warp has several rows, so that the loads of the next row, the two buffers
of sums in turn and the stages of bulk copies all come round; in place and not.

Bounds: those of test_norm, which go by a row.  dweight: a warp has at most 6 rows (20000 rows, 8 a block, 456 blocks), then 8
warps, 15 of 456 blocks one after another and 5 steps: 34 * 2^-24 of the sum of |terms|, less than the 2^-17 - 2^-19 there."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_util import randn
from test_norm import BF, F32, HALF, backward64, check_rows, check_y, forward64, make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("residual", [None, BF, F32])
@pytest.mark.parametrize("rows,H", [(20000, 256), (20000, 1000), (3001, 1032), (3001, 7168), (700, 16384)])
def test_forward(rows, H, residual):
    x, r, w, _ = make(rows, H, residual, F32, rows + H)
    fp8 = H % 128 == 0
    got = ep.rms_norm(x, w, 1e-5, residual=r, fp8=fp8)
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    if r is not None:
        assert torch.equal(got["residual"], h)
    n, _ = forward64(h, w, 1e-5)
    check_y(got["y"], n)
    if fp8:
        check_rows(got["rows"], n)
    del n
    out = {"y": x} | ({} if r is None else {"residual": r})
    same = ep.rms_norm(x, w, 1e-5, residual=r, fp8=fp8, out=out)
    assert same["y"] is x and torch.equal(x, got["y"]) and (r is None or torch.equal(r, got["residual"]))
    assert not fp8 or torch.equal(same["rows"][:, :H + H // 32], got["rows"][:, :H + H // 32])


@gpu
@pytest.mark.parametrize("kind,dres", [(BF, True), (BF, False), (F32, True)])
@pytest.mark.parametrize("rows,H", [(20000, 256), (20000, 1000), (3001, 1032), (2000, 7168), (500, 16384)])
def test_backward(rows, H, kind, dres):
    h, _, w, g = make(rows, H, None, F32, rows + 2 * H)
    h = (2 * h.float()).to(kind)
    dy = randn((rows, H), g).to(BF)
    d = randn((rows, H), g).to(kind) if dres else None
    dx, dw = ep.rms_norm_backward(dy, h, w, 1e-5, dresidual=d)
    ref, mag, dw64, dwmag = backward64(dy, h, w, d, 1e-5)
    assert ((dx.double() - ref).abs() <= HALF[kind] * ref.abs() + 2.0 ** -18 * mag).all()
    assert ((dw.double() - dw64).abs() <= 2.0 ** -17 * dwmag).all()
    over = d if dres else torch.full_like(dx, 9.0)              # the rows' own memory, read before it is written, or a new one
    again, dw2 = ep.rms_norm_backward(dy, h, w, 1e-5, dresidual=d, out=(over, torch.full_like(dw, 9.0)))
    assert again is over and torch.equal(over, dx) and torch.equal(dw2, dw)
