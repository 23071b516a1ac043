"""Pairs of blocks over many tiles each: every ring of barriers comes round several times, and launches that follow one another at
once have other rows and weights, so that codes or scales of a stage, a tile or a launch before would show.  Bounds: test_fp4's."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from expert_shapes import form_launched, sms
from expert_util import assert_bf16_close, gen
from test_experts import groups_of
from test_fp4 import BF, assert_fp4_close, product64, rows4, swiglu64, values4, weight4


def tiles_a_pair(counts, columns):
    return sum(-(-c // 256) for c in counts) * columns / (sms() // 2)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,K,I", [([1300, 1025, 1536, 1100], 640, 2816), ([1290, 1400, 1536, 1111], 1536, 2816), ([5000], 128, 4096)])
def test_first_product(counts, K, I):
    cnt, off, hoff, rows = groups_of(counts, 2)
    G = len(counts)
    assert tiles_a_pair(counts, -(-I // 96)) > 8              # the ring of announced tiles has four slots
    sets = []
    for seed in (1, 2):
        g = gen(seed)
        x, xs = rows4(rows, K, g)
        w, ws = weight4(G, 2 * I, K, g)
        sets.append((x, xs + (seed - 1) * 3, w, ws))            # the second's scales are 8 times as large
    out = [tuple(torch.full((rows, n), 7, dtype=torch.uint8, device="cuda") for n in (I // 2, I // 32)) for _ in range(6)]
    call = lambda s, o, stream=None: ep.expert_swiglu_fp4(*s, counts=cnt, offsets=off, out=o, expected_rows=max(counts), stream=stream)  # noqa: E731
    assert form_launched(lambda stream: call(sets[0], out[0], stream)) == "pairs"
    for i, o in enumerate(out):
        call(sets[i % 2], o)
    for i, (x, xs, w, ws) in enumerate(sets):
        assert all(torch.equal(a, b) for o in out[i + 2::2] for a, b in zip(o, out[i]))
        for e, (o, c) in enumerate(zip(hoff, counts)):
            s = slice(o, o + c)
            assert_fp4_close(out[i][0][s], out[i][1][s], *swiglu64(values4(x[s], xs[s]), values4(w[e], ws[e])))


@pytest.mark.gpu
@pytest.mark.parametrize("counts,K,N", [([1536, 1301, 1100, 1536], 640, 6720), ([1536, 1290, 1111, 1400], 1536, 6731), ([4352], 128, 9100), ([4300], 1664, 9184)])
def test_second_product(counts, K, N):
    cnt, off, hoff, rows = groups_of(counts, 2)
    G = len(counts)
    assert tiles_a_pair(counts, -(-N // 224)) > 8
    sets = []
    for seed in (3, 4):
        g = gen(seed)
        x, xs = rows4(rows, K, g)
        w, ws = weight4(G, N, K, g)
        sets.append((x, xs + (seed - 3) * 3, w, ws))
    out = [torch.full((rows, N), 7.0, dtype=BF, device="cuda") for _ in range(6)]
    call = lambda s, o, stream=None: ep.expert_gemm_fp4(*s, counts=cnt, offsets=off, out=o, expected_rows=max(counts), stream=stream)  # noqa: E731
    assert form_launched(lambda stream: call(sets[0], out[0], stream)) == "pairs"
    for i, o in enumerate(out):
        call(sets[i % 2], o)
    for i, (x, xs, w, ws) in enumerate(sets):
        assert all(torch.equal(o, out[i]) for o in out[i + 2::2])
        for e, (o, c) in enumerate(zip(hoff, counts)):
            s = slice(o, o + c)
            assert_bf16_close(out[i][s], *product64(values4(x[s], xs[s]), values4(w[e], ws[e])), f"group {e}")
