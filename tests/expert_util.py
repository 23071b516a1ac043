"""Inputs, the 64-bit reference and the error bounds of the expert operators' tests.

The bounds are worst-case sums of roundings, not observed errors.  An fp32 sum
of a product of K terms: every 128-block is four tensor-core steps and one
fused multiply-add, so with S = sum |x||w| its error is at most
(K/128 + 8) * 2^-23 * S (each addition rounds or truncates at 2^-23 of a
partial sum that S bounds); bf16 rounding adds 2^-9 of the result, held to 2^-8.
"""
import torch

U = 2.0 ** -23


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def quantize_rows(v):
    """e4m3 codes and scales per 128 channels of fp32 rows [..][K]."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    s = b.abs().amax(-1) / 448.0
    q = torch.where(s[..., None] > 0, b / s[..., None], b).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(v.shape), s


def quantize_weight(w):
    """e4m3 codes and scales per 128 x 128 block of fp32 weights [G][N][K]."""
    G, N, K = w.shape
    nb = -(-N // 128)
    p = torch.zeros(G, nb * 128, K, device="cuda")
    p[:, :N] = w
    b = p.view(G, nb, 128, K // 128, 128)
    s = (b.abs().amax((2, 4)) / 448.0).clamp(min=1e-30)
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(G, nb * 128, K)[:, :N]
    return q.contiguous(), s.contiguous()


def rows64(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(128, -1)


def weight64(codes, scales):
    """One group's weight [N][K] (bf16, or codes and scales)."""
    if scales is None:
        return codes.double()
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(128, 0)[: v.shape[0]].repeat_interleave(128, 1)


def product64(x, w):
    """(y, bound of the fp32 sum's error) of rows [m][K] and a weight [N][K] in 64 bits."""
    y = x @ w.t()
    s = x.abs() @ w.abs().t()
    return y, (x.shape[1] // 128 + 8) * U * s


def silu64(g):
    return g / (1 + torch.exp(-g))


def swiglu64(x, w13):
    """(h, bound of its error in fp32): |silu'| <= 1.1, and 2^-20 covers exp, the division and the product."""
    n = w13.shape[0] // 2
    y, e = product64(x, w13)
    g, u = y[:, :n], y[:, n:]
    h = silu64(g) * u
    return h, 1.1 * e[:, :n] * u.abs() + silu64(g).abs() * e[:, n:] + 1.1 * e[:, :n] * e[:, n:] + 2.0 ** -20 * h.abs()


def assert_bf16_close(got, ref, err, what=""):
    d = (got.double() - ref).abs()
    lim = 2.0 ** -8 * ref.abs() + err + 1e-38
    bad = ~(d <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside the bound, worst {float((d / lim).max()):.3g} of it"


def assert_fp8_close(codes, scales, h, err, what=""):
    """Codes and scales of h: the scale within its block's largest error, the value within half a step of e4m3
    (2^-4 of it, or 2^-10 of the scale among subnormals) and twice the error."""
    amax = h.abs().reshape(h.shape[0], -1, 128).amax(-1)
    emax = err.reshape(h.shape[0], -1, 128).amax(-1)
    ds = (scales.double() - amax / 448).abs()
    assert (ds <= emax / 448 + 2 * U * amax / 448 + 1e-44).all(), f"{what}: scales off by {float((ds / (amax / 448)).max()):.3g}"
    got = rows64(codes, scales)
    step = scales.double().repeat_interleave(128, -1) * 2.0 ** -10
    lim = 2.0 ** -4 * (h.abs() + err) + step + 2 * err + 2.0 ** -20 * h.abs() + 1e-44
    d = (got - h).abs()
    assert (d <= lim).all(), f"{what}: {int((d > lim).sum())} codes outside the bound, worst {float((d / lim).max()):.3g}"
