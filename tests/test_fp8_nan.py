"""The FP8 codec and NaN: a NaN channel has a NaN code, also where its block holds nothing but zeros beside it."""
import numpy as np
import pytest
import torch

import oracle as orc
from combine_get_dispatch_histograms_gb300 import Context, LLBuffer, inputs
from parity_util import bits, eq

QNAN, NEG_QNAN = 0x7FC0, 0xFFC0


def rows_with_nan(T, H, seed):
    """bf16 bits [T][H]: blocks of nothing but NaN, of zeros and a NaN, and NaN among finite values (of both signs)."""
    xb = bits(inputs.random_x(1, T, H, seed)).reshape(T, H).copy()
    xb[0] = QNAN
    xb[1, :128], xb[1, 5] = 0, QNAN
    xb[2, 128:256], xb[2, 130], xb[2, 131] = 0x8000, NEG_QNAN, 0
    xb[3, 7] = QNAN
    return xb


def test_the_oracle_keeps_a_nan():
    xb = rows_with_nan(4, 256, 1)
    c0, s0 = orc.quantize_row(xb[0])
    assert (s0 == 0).all() and (c0 == 0x7F).all()
    c1, s1 = orc.quantize_row(xb[1])
    assert s1[0] == 0 and c1[5] == 0x7F and (np.delete(c1[:128], 5) == 0).all() and s1[1] > 0
    c2, s2 = orc.quantize_row(xb[2])
    assert s2[1] == 0 and c2[130] == 0xFF and c2[131] == 0 and (c2[132:] == 0x80).all()
    c3, s3 = orc.quantize_row(xb[3])
    assert s3[0] > 0 and c3[7] & 0x7F == 0x7F


@pytest.mark.gpu
def test_quantised_rows_and_messages_keep_a_nan():
    T, H = 6, 256
    xb = rows_with_nan(T, H, 2)
    x = torch.from_numpy(xb.view(np.int16)).view(torch.bfloat16).reshape(1, T, H).cuda()
    want = np.stack([np.concatenate([c, s.view(np.uint8)]) for c, s in map(orc.quantize_row, xb)])
    ctx = Context(1, 1, 1, T, H, num_channels=1)
    idx, w = torch.zeros(1, T, 1, dtype=torch.int64, device="cuda"), torch.ones(1, T, 1, device="cuda")
    h = ctx.notify_dispatch(idx, ctx.get_dispatch_layout(idx))
    eq(bits(ctx.quantize_fp8(x))[:, :H + H // 32], want, "fp8 rows")
    eq(bits(ctx.dispatch_permuted_quant(x, idx, w, h)["permuted_xq"])[:, :H + H // 32], want, "quantised in the dispatch")
    ctx.check()
    buf = LLBuffer(1, 1, 1, T, H, T)
    pk = buf.dispatch(x, idx)
    buf.check()
    eq(pk["packed_x"][0, 0, :T], want[:, :H], "message codes")
    eq(pk["packed_scales"][0, 0, :T], want[:, H:].view(np.float32), "message scales")
