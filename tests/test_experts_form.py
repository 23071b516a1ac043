"""Which form of the product kernel a call takes, as its launch is recorded in a graph: for speed alone, so results do not show it."""
import pytest
import torch

import combine_get_dispatch_histograms_gb300 as ep
from combine_get_dispatch_histograms_gb300 import LLBuffer, inputs
from expert_shapes import form_launched, form_of

gpu = pytest.mark.gpu


def arrays(G, rows, K, N):
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, xs = z(*rows, K), z(*rows, K // 128, dtype=torch.float32)
    w, ws = z(G, N, K), z(G, -(-N // 128), K // 128, dtype=torch.float32)
    return x, xs, w, ws, z(*rows, N, dtype=torch.bfloat16), (z(*rows, N // 2), z(*rows, N // 256, dtype=torch.float32))


def both(x, xs, w, ws, out, hidden, **kw):
    one = form_launched(lambda s: ep.expert_gemm(x, xs, w, ws, out=out, stream=s, **kw))
    assert form_launched(lambda s: ep.expert_swiglu(x, xs, w, ws, out=hidden, stream=s, **kw)) == one
    return one


@gpu
@pytest.mark.parametrize("m,form", [(64, "one"), (128, "one"), (129, "pairs"), (256, "pairs"), (257, "one"), (384, "one"), (385, "pairs"),
                                    (512, "pairs"), (513, "one"), (640, "one"), (641, "pairs"), (896, "pairs"), (1025, "pairs")])
def test_by_the_rows_of_a_group(m, form):
    """What the arrays hold, shared out, or what the caller expects: pairs where they need 1.75 times fewer tiles or better."""
    G, K, N = 40, 256, 1024
    a = arrays(G, (G * m,), K, N)
    cnt = torch.full((G,), m, dtype=torch.int32, device="cuda")
    off = torch.arange(0, G * m, m, dtype=torch.int32, device="cuda")
    assert both(*a, counts=cnt, offsets=off) == form == form_of(G * m, G, N, K)
    a = arrays(G, (G * 700,), K, N)
    assert both(*a, counts=cnt, offsets=off, expected_rows=m) == form == form_of(G * 700, G, N, K, m)


@gpu
@pytest.mark.parametrize("cap,full,counted", [(200, "pairs", "one"), (1024, "pairs", "one"), (2048, "pairs", "one"), (4096, "pairs", "pairs"),
                                              (64, "one", "one"), (300, "one", "one")])
def test_regions(cap, full, counted):
    """Without counts every row of a region counts; with counts a region is taken as filled to a sixteenth."""
    G, K, N = 40, 128, 512
    a = arrays(G, (G, cap), K, N)
    assert both(*a) == full
    cnt = torch.full((G,), cap, dtype=torch.int32, device="cuda")
    assert both(*a, counts=cnt) == counted
    assert both(*a, counts=cnt, expected_rows=cap) == full


@gpu
@pytest.mark.parametrize("rows,N,K", [(1, 4096, 7168), (64, 512, 1024), (777, 1024, 1408)])
def test_few_tiles_share_their_k(rows, N, K):
    x, xs, w, ws, out, hidden = arrays(1, (rows,), K, N)
    assert both(x, xs, w[0], ws[0], out, hidden) == "cluster" == form_of(rows, 1, N, K)


@gpu
def test_a_microbatch_expects_its_own_tokens():
    R, E, K, T, H, I = 4, 8, 2, 256, 256, 512
    buf = LLBuffer(R, E, K, T, H, T)
    x, idx = inputs.random_x(R, T, H, 1).cuda(), inputs.random_topk(R, E, K, T, 3).cuda()
    _, w, ws, y, hidden = arrays(E, (E, R * T), H, 2 * I)[1:]
    _, w2, w2s, y, _ = arrays(E, (E, R * T), I, 1024)[1:]
    packed = buf.dispatch(x, idx, 0, 64)
    for n, form in ((None, "pairs"), (64, "one"), (128, "one"), (200, "pairs")):      # 256, 64, 128, 200 rows an expert
        assert form_launched(lambda s: buf.expert_swiglu(packed, w, ws, out=hidden, stream=s, n=n)) == form
        assert form_launched(lambda s: buf.expert_gemm(hidden, packed, w2, w2s, out=y, stream=s, n=n)) == form
    buf.check()
