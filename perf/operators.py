"""Cases for the expert operators: the FP8 expert products and the whole layer for a few tokens.

Three operators, over the sizes that dispatch and combine are used with:

* ``gemm``    y = x w^T per expert, e4m3 codes with a scale per 128 channels (x) and per 128 x 128 block (w);
* ``swiglu``  h = silu(x wg^T) * (x wu^T) per expert, h again e4m3 codes with a scale per 128 channels;
* ``tokens``  the whole layer (both products, activation, weighted sum over the top-k) for up to 64 tokens.

``own`` selects the framework's calls; otherwise the plain form runs: elementary torch operations in 32 bits,
rounded once at the end.  Rows of ``gemm`` and ``swiglu`` come in the three layouts a user has: ``permuted``
(dispatch into per-expert blocks, FP8 rows with their scales behind the codes), ``packed`` (the low-latency
receive, fixed regions per expert with counts) and ``dense`` (one weight for all rows).
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


def listed():
    return [
        # the smallest dispatch of the framework: a few rows per expert, launch latency counts
        {"name": "gemm tiny", "op": "gemm", "layout": "permuted", "experts": 8, "topk": 2, "tokens": 64, "k": 128, "n": 128,
         "skew": 0.0, "mask": 0.0},
        # one token through one FP8 projection: the weight is read once for a single row
        {"name": "gemm one row", "op": "gemm", "layout": "dense", "experts": 1, "topk": 1, "tokens": 1, "k": 7168, "n": 4096,
         "skew": 0.0, "mask": 0.0},
        # a dense product whose rows and columns fill no tile
        {"name": "gemm odd", "op": "gemm", "layout": "dense", "experts": 1, "topk": 1, "tokens": 777, "k": 1408, "n": 1099,
         "skew": 0.0, "mask": 0.0},
        # second product of a low-latency decode step: 16 ranks x 128 tokens, about 64 rows per expert region
        {"name": "gemm decode", "op": "gemm", "layout": "packed", "experts": 256, "topk": 8, "tokens": 2048, "k": 2048, "n": 7168,
         "skew": 0.0, "mask": 0.0},
        # second product of a prefill step: 8 ranks x 4096 tokens, popular and unpopular experts
        {"name": "gemm prefill", "op": "gemm", "layout": "permuted", "experts": 256, "topk": 8, "tokens": 32768, "k": 2048,
         "n": 7168, "skew": 0.5, "mask": 0.0},
        # first product of a small ragged batch: many experts get one row or none
        {"name": "swiglu ragged", "op": "swiglu", "layout": "permuted", "experts": 64, "topk": 4, "tokens": 37, "k": 640, "n": 384,
         "skew": 0.5, "mask": 0.05},
        # first product of the low-latency decode step
        {"name": "swiglu decode", "op": "swiglu", "layout": "packed", "experts": 256, "topk": 8, "tokens": 2048, "k": 7168,
         "n": 2048, "skew": 0.0, "mask": 0.0},
        # first product of a large batch with few very popular experts, 5 % of the entries masked
        {"name": "swiglu skewed", "op": "swiglu", "layout": "permuted", "experts": 256, "topk": 8, "tokens": 65536, "k": 4096,
         "n": 1408, "skew": 1.5, "mask": 0.05},
        # one token, the smallest layer: latency
        {"name": "layer tiny", "op": "tokens", "weights": "fp8", "experts": 8, "topk": 2, "tokens": 1, "k": 128, "n": 128,
         "skew": 0.0, "mask": 0.0},
        # one token of a large layer: eight experts' weights
        {"name": "layer one token", "op": "tokens", "weights": "fp8", "experts": 256, "topk": 8, "tokens": 1, "k": 7168, "n": 2048,
         "skew": 0.0, "mask": 0.0},
        # a small batch with bf16 weights and masked entries
        {"name": "layer bf16 batch", "op": "tokens", "weights": "bf16", "experts": 256, "topk": 8, "tokens": 17, "k": 4096,
         "n": 1408, "skew": 0.5, "mask": 0.05},
        # the largest batch the few-token layer takes: most experts, some with many tokens
        {"name": "layer full batch", "op": "tokens", "weights": "fp8", "experts": 256, "topk": 8, "tokens": 64, "k": 7168,
         "n": 2048, "skew": 1.0, "mask": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["gemm", "swiglu", "tokens"])
        c = {"op": op, "k": BLOCK * _log(rng, 1, 56), "skew": rng.choice([0.0, 0.5, 1.0, 1.5]), "mask": rng.choice([0.0, 0.05, 0.3])}
        if op == "tokens":
            c["weights"] = rng.choice(["fp8", "bf16"])
            c["tokens"] = _log(rng, 1, 64)
            c["n"] = BLOCK * _log(rng, 1, 16)
        else:
            c["layout"] = rng.choice(["permuted", "packed", "dense"])
            c["tokens"] = _log(rng, 1, 32768 if c["layout"] == "permuted" else 4096)
            c["n"] = _log(rng, 1, 7168) if op == "gemm" else BLOCK * _log(rng, 1, 16)
        if c.get("layout") == "dense":
            c["experts"], c["topk"], c["skew"], c["mask"] = 1, 1, 0.0, 0.0
        else:
            c["experts"] = _log(rng, 4, 256)
            c["topk"] = rng.randint(1, min(8, c["experts"]))
        if c["tokens"] * c["topk"] < 16:  # so few that a mask could leave nothing at all
            c["mask"] = 0.0
        if 3072 in (c["k"], c["n"], 2 * c["n"], c["tokens"], c["tokens"] * c["topk"]):
            continue
        if c["experts"] * c["k"] * c["n"] <= 256 * 7168 * 2048 and work(c)["flops"] <= 7e12:
            return c


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _quantize_weight(experts, n, k, g):
    """e4m3 codes [experts][n][k] of normal weights and their scales [experts][ceil(n/128)][k/128]."""
    nb = -(-n // BLOCK)
    codes = torch.empty(experts, n, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, nb, k // BLOCK, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (nb * BLOCK * k))
    for i in range(0, experts, step):
        e = min(step, experts - i)
        w = torch.zeros(e, nb * BLOCK, k, dtype=torch.float32, device="cuda")
        w[:, :n] = _normal((e, n, k), g) * k ** -0.5
        w = w.view(e, nb, BLOCK, k // BLOCK, BLOCK)
        s = w.abs().amax(dim=(2, 4)) / E4M3_MAX
        q = (w / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[i:i + e] = q.view(e, nb * BLOCK, k)[:, :n]
        scales[i:i + e] = s
    return codes, scales


def _bf16_weight(experts, n, k, g):
    w = torch.empty(experts, n, k, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for i in range(0, experts, step):
        e = min(step, experts - i)
        w[i:i + e] = (_normal((e, n, k), g) * k ** -0.5).to(torch.bfloat16)
    return w


def _routing(c, g):
    """topk_idx [tokens][topk] int64 (-1 masked) and the weights, softmax over the chosen."""
    logits = _normal((c["tokens"], c["experts"]), g) + c["skew"] * _normal((c["experts"],), g)
    vals, idx = torch.topk(logits, c["topk"], dim=1)
    drop = torch.rand(idx.shape, generator=g, device="cuda") < c["mask"]
    return torch.where(drop, -1, idx), torch.softmax(vals, dim=1)


def _rows(rows, k, activation, g):
    """FP8 rows [rows][k + k/32]: e4m3 codes, then k/128 fp32 scales."""
    pad = (k + k // 32 + 15) // 16 * 16
    out = torch.zeros(rows, pad, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // k)
    for i in range(0, rows, step):
        m = min(step, rows - i)
        v = _normal((m, k), g)
        if activation:  # what the first product hands on: silu(gate) * up
            v = v * torch.sigmoid(v) * _normal((m, k), g)
        v = v.to(torch.bfloat16).float().view(m, k // BLOCK, BLOCK)
        s = v.abs().amax(dim=2) / E4M3_MAX
        out[i:i + m, :k] = (v / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(m, k)
        out[i:i + m, k:k + k // 32] = s.view(torch.uint8)
    return out


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx, wts = _routing(c, g)
    if c["op"] == "tokens":
        s = {"case": c, "x": _normal((c["tokens"], c["k"]), g).to(torch.bfloat16), "topk_idx": idx, "topk_weights": wts,
             "w13_scales": None, "w2_scales": None}
        if c["weights"] == "fp8":
            s["w13"], s["w13_scales"] = _quantize_weight(c["experts"], 2 * c["n"], c["k"], g)
            s["w2"], s["w2_scales"] = _quantize_weight(c["experts"], c["k"], c["n"], g)
        else:
            s["w13"] = _bf16_weight(c["experts"], 2 * c["n"], c["k"], g)
            s["w2"] = _bf16_weight(c["experts"], c["k"], c["n"], g)
        return s
    k, n, gemm = c["k"], c["n"], c["op"] == "gemm"
    s = {"case": c}
    s["w"], s["w_scales"] = _quantize_weight(c["experts"], n if gemm else 2 * n, k, g)
    counts = torch.bincount(idx[idx >= 0], minlength=c["experts"]).to(torch.int32)
    if c["layout"] == "packed":  # regions of a fixed size, rows past the count unused
        cap = c["tokens"]
        s["host_counts"] = counts.tolist()
        s["host_offsets"] = [cap * e for e in range(c["experts"])]
        rows = _rows(c["experts"] * cap, k, gemm, g)
        s["x"] = rows[:, :k].contiguous().view(c["experts"], cap, k)
        s["x_scales"] = rows[:, k:k + k // 32].contiguous().view(torch.float32).view(c["experts"], cap, k // BLOCK)
        s["counts"], s["offsets"] = counts, None
        total = c["experts"] * cap
    else:
        s["host_counts"] = counts.tolist()
        s["host_offsets"] = (torch.cumsum(counts, 0) - counts).tolist()
        total = c["tokens"] * c["topk"]  # the worst case, whatever is masked; rows past the groups unused
        rows = _rows(total, k, gemm, g)
        s["x"] = rows[:, :k]
        s["x_scales"] = rows[:, k:k + k // 32].view(torch.float32)
        s["counts"] = counts
        s["offsets"] = (torch.cumsum(counts, 0) - counts).to(torch.int32)
        if c["layout"] == "dense":
            s["w"], s["w_scales"], s["counts"], s["offsets"] = s["w"][0], s["w_scales"][0], None, None
    lead = (c["experts"], c["tokens"]) if c["layout"] == "packed" else (total,)
    if gemm:  # the buffer that a serving loop keeps; rows of no group stay zero
        s["out"] = torch.zeros(*lead, n, dtype=torch.bfloat16, device="cuda")
    else:
        s["out"] = torch.zeros(*lead, n, dtype=torch.uint8, device="cuda")
        s["out_scales"] = torch.zeros(*lead, n // BLOCK, dtype=torch.float32, device="cuda")
    return s


def _values(codes, scales):
    """What e4m3 codes [r][k] with a scale per 128 channels stand for."""
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.view(*v.shape[:-1], -1, BLOCK) * scales[..., None]).view(v.shape)


def _weight_values(codes, scales):
    """What e4m3 codes [...][n][k] with a scale per 128 x 128 block stand for (bf16 weights: themselves)."""
    if scales is None:
        return codes.float()
    n, k = codes.shape[-2:]
    s = scales[..., torch.arange(n, device="cuda") // BLOCK, :]
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.view(*v.shape[:-1], k // BLOCK, BLOCK) * s[..., None]).view(v.shape)


def _quantize(h):
    v = h.view(h.shape[0], -1, BLOCK)
    s = v.abs().amax(dim=2) / E4M3_MAX
    q = torch.where(s[:, :, None] > 0, v / s[:, :, None], v).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(h.shape), s


def _plain_rows(s):
    c = s["case"]
    k, n = c["k"], c["n"]
    x, xs = s["x"].reshape(-1, k), s["x_scales"].reshape(-1, k // BLOCK)
    w, ws = s["w"].view(c["experts"], -1, k), s["w_scales"].view(c["experts"], -1, k // BLOCK)
    for e in range(c["experts"]):  # ragged groups: one product each
        lo, m = s["host_offsets"][e], s["host_counts"][e]
        if m == 0:
            continue
        y = _values(x[lo:lo + m], xs[lo:lo + m]) @ _weight_values(w[e], ws[e]).t()
        if c["op"] == "gemm":
            s["out"].view(-1, n)[lo:lo + m] = y.to(torch.bfloat16)
        else:
            gate, up = y[:, :n], y[:, n:]
            q, sc = _quantize(gate * torch.sigmoid(gate) * up)
            s["out"].view(-1, n)[lo:lo + m] = q
            s["out_scales"].view(-1, n // BLOCK)[lo:lo + m] = sc
    return _outputs(s)


def _outputs(s):
    if s["case"]["op"] == "gemm":
        return s["out"]
    return {"h": s["out"].view(torch.float8_e4m3fn), "scales": s["out_scales"]}


def _plain_tokens(s):
    c = s["case"]
    x = s["x"].float()
    out = torch.zeros_like(x)
    scale = lambda name, e: None if s[name] is None else s[name][e]  # noqa: E731
    for j in range(c["topk"]):  # one choice of every token at a time: its experts' weights gathered
        e = s["topk_idx"][:, j].clamp(min=0)
        w = torch.where(s["topk_idx"][:, j] >= 0, s["topk_weights"][:, j], 0.0)
        y = torch.bmm(_weight_values(s["w13"][e], scale("w13_scales", e)), x[:, :, None])[:, :, 0]
        gate, up = y[:, :c["n"]], y[:, c["n"]:]
        h = gate * torch.sigmoid(gate) * up
        out += w[:, None] * torch.bmm(_weight_values(s["w2"][e], scale("w2_scales", e)), h[:, :, None])[:, :, 0]
    return out.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        return _plain_tokens(state) if c["op"] == "tokens" else _plain_rows(state)
    import combine_get_dispatch_histograms_gb300 as ep
    if c["op"] == "tokens":
        return ep.moe_tokens(state["x"], state["topk_idx"], state["topk_weights"], state["w13"], state["w2"],
                             w13_scales=state["w13_scales"], w2_scales=state["w2_scales"])
    if c["op"] == "gemm":
        ep.expert_gemm(state["x"], state["x_scales"], state["w"], state["w_scales"], counts=state["counts"],
                       offsets=state["offsets"], out=state["out"])
    else:
        ep.expert_swiglu(state["x"], state["x_scales"], state["w"], state["w_scales"], counts=state["counts"],
                         offsets=state["offsets"], out=(state["out"], state["out_scales"]))
    return _outputs(state)


def _pairs(c):
    """Expected (token, choice) pairs and experts with at least one (skewed routing reaches fewer: this is an estimate)."""
    pairs = c["tokens"] * c["topk"] * (1.0 - c["mask"])
    hit = c["experts"] * (1.0 - (1.0 - c["topk"] * (1.0 - c["mask"]) / c["experts"]) ** c["tokens"]) if c["experts"] > 1 else 1.0
    return pairs, max(1.0, hit)


def work(case):
    c = case
    k, n = c["k"], c["n"]
    pairs, hit = _pairs(c)
    if c["op"] == "tokens":
        per = 2.0 if c["weights"] == "bf16" else 1.0 + 4.0 / BLOCK ** 2
        return {"bytes": hit * 3 * n * k * per + c["tokens"] * (4 * k + 12 * c["topk"]), "flops": 6.0 * pairs * n * k}
    weight = hit * (n if c["op"] == "gemm" else 2 * n) * k * (1 + 4.0 / BLOCK ** 2)
    if c["op"] == "gemm":
        return {"bytes": pairs * (k + k / 32 + 2 * n) + weight, "flops": 2.0 * pairs * n * k}
    return {"bytes": pairs * (k + k / 32 + n + n / 32) + weight, "flops": 4.0 * pairs * n * k}


def _table():
    """The 256 values of e4m3 in 64 bits, from its definition."""
    t = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t.append(-v if b & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device="cuda")


def exact(case, seed):
    c = dict(case)
    if work(c)["flops"] > 1.4e13:
        return None
    s = prepare(case, seed)
    table = _table()
    n, k = c["n"], c["k"]

    def matrix(codes, scales):  # the weight of one expert, each code times its block's scale
        if scales is None:
            return codes.double()
        rows, cols = codes.shape
        spread = scales.double().repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
        return table[codes.int()] * spread

    if c["op"] == "tokens":
        out = torch.zeros(c["tokens"], k, dtype=torch.float64, device="cuda")
        for e in torch.unique(s["topk_idx"]).tolist():
            if e < 0:
                continue
            t, j = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
            w13 = matrix(s["w13"][e], None if s["w13_scales"] is None else s["w13_scales"][e])
            w2 = matrix(s["w2"][e], None if s["w2_scales"] is None else s["w2_scales"][e])
            y = torch.einsum("tk,nk->tn", s["x"][t].double(), w13)
            h = y[:, :n] / (1 + torch.exp(-y[:, :n])) * y[:, n:]
            out.index_add_(0, t, s["topk_weights"][t, j].double()[:, None] * torch.einsum("tn,kn->tk", h, w2))
        return out
    x = s["x"].reshape(-1, k)
    xs = s["x_scales"].reshape(-1, k // BLOCK)
    w, ws = s["w"].view(c["experts"], -1, k), s["w_scales"].view(c["experts"], -1, k // BLOCK)
    first = torch.zeros(x.shape[0], n, dtype=torch.float64, device="cuda")
    scales = None if c["op"] == "gemm" else torch.zeros(x.shape[0], n // BLOCK, dtype=torch.float64, device="cuda")
    for e, (lo, m) in enumerate(zip(s["host_offsets"], s["host_counts"])):
        if m == 0:
            continue
        y = torch.einsum("rk,nk->rn", table[x[lo:lo + m].int()] * xs[lo:lo + m].double().repeat_interleave(BLOCK, 1), matrix(w[e], ws[e]))
        if c["op"] == "gemm":
            first[lo:lo + m] = y
        else:  # the value that each code rounds, and the block's scale
            h = y[:, :n] / (1 + torch.exp(-y[:, :n])) * y[:, n:]
            a = h.view(m, -1, BLOCK).abs().amax(dim=2) / E4M3_MAX
            scales[lo:lo + m] = a
            first[lo:lo + m] = h / a.clamp(min=1e-300).repeat_interleave(BLOCK, 1)
    if c["op"] == "gemm":
        return first.view(s["out"].shape)
    return {"h": first.view(s["out"].shape), "scales": scales.view(s["out_scales"].shape)}
