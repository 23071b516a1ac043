"""Cases for the operators around dispatch: the norm before it, the router with its balance loss, and 4-bit experts.

* ``norm``     h = x + residual, RMS norm of h, out as bf16 and as FP8 rows; ``grad``: its backward pass too;
* ``route``    router logits to topk_idx and topk_weights;
* ``balance``  the balance loss with per-expert counts and the gradient of the logits; ``route``: the training step of a
  router, choice, loss and both gradients at once;
* ``linear4``  bf16 rows quantised to MXFP4 and multiplied by an MXFP4 weight;
* ``experts4`` both products of a layer's experts on dispatched MXFP4 rows, with SwiGLU and requantisation between.

``own`` selects the framework's calls; otherwise the plain form runs: elementary torch operations in 32 bits, rounded
once at the end.  MXFP4: two e2m1 codes a byte (the lower channel in the lower half), one E8M0 exponent per 32 channels.
"""
import math

import torch

own = False

EPS = 1e-6
COEF = 0.01


def listed():
    return [
        # one token of a decode step of a large model: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "hidden": 7168, "residual": "bf16", "weight": "bf16", "fp8": True,
         "grad": False},
        # a prefill step, 8 ranks x 4096 tokens: the norm before the layer, with what the router and what dispatch read
        {"name": "norm prefill", "op": "norm", "rows": 32768, "hidden": 7168, "residual": "bf16", "weight": "bf16", "fp8": True,
         "grad": False},
        # a training batch with odd sizes and a residual stream in 32 bits: forward and backward
        {"name": "norm train odd", "op": "norm", "rows": 4099, "hidden": 4104, "residual": "fp32", "weight": "fp32", "fp8": False,
         "grad": True},
        # a training batch of a large model
        {"name": "norm train", "op": "norm", "rows": 16384, "hidden": 7168, "residual": "bf16", "weight": "fp32", "fp8": False,
         "grad": True},
        # a low-latency decode step, 16 ranks x 128 tokens
        {"name": "route decode", "op": "route", "tokens": 2048, "experts": 256, "topk": 8, "logits": "bf16", "scoring": "softmax",
         "normalize": True, "bias": False, "groups": 1, "topk_groups": 1, "closed": 0, "skew": 0.0, "mask": 0.0},
        # a prefill step over 8 nodes' experts, 4 nodes a token, with the bias of a balanced router
        {"name": "route prefill", "op": "route", "tokens": 32768, "experts": 256, "topk": 8, "logits": "fp32", "scoring": "sigmoid",
         "normalize": True, "bias": True, "groups": 8, "topk_groups": 4, "closed": 0, "skew": 0.5, "mask": 0.0},
        # a few short sequences over few experts
        {"name": "balance small", "op": "balance", "sequences": 4, "tokens": 40, "experts": 8, "topk": 2, "logits": "fp32",
         "scoring": "softmax", "normalize": True, "route": False, "closed": 0, "skew": 0.5, "mask": 0.1},
        # a training step's router: 32 sequences, popular experts, a few padded tokens, choice, loss and gradients
        {"name": "balance train", "op": "balance", "sequences": 32, "tokens": 2048, "experts": 256, "topk": 8, "logits": "fp32",
         "scoring": "softmax", "normalize": True, "route": True, "closed": 0, "skew": 1.0, "mask": 0.05},
        # one token through one projection in 4 bits
        {"name": "linear4 one row", "op": "linear4", "rows": 1, "k": 7168, "n": 4096},
        # rows and columns that fill no tile
        {"name": "linear4 odd", "op": "linear4", "rows": 777, "k": 1408, "n": 1099},
        # the experts of a decode step, 16 ranks x 128 tokens: about 64 rows an expert
        {"name": "experts4 decode", "op": "experts4", "experts": 256, "topk": 8, "tokens": 2048, "k": 7168, "n": 2048, "skew": 0.0,
         "mask": 0.0},
        # the experts of a prefill step, 8 ranks x 1024 tokens, popular and unpopular ones
        {"name": "experts4 prefill", "op": "experts4", "experts": 256, "topk": 8, "tokens": 8192, "k": 7168, "n": 2048, "skew": 0.5,
         "mask": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "route", "balance", "linear4", "experts4"])
        c = {"op": op}
        if op == "norm":
            c |= {"rows": _log(rng, 1, 32768), "residual": rng.choice(["none", "bf16", "fp32"]), "weight": rng.choice(["bf16", "fp32"]),
                  "fp8": rng.random() < 0.5, "grad": rng.random() < 0.5}
            c["hidden"] = 128 * _log(rng, 1, 128) if c["fp8"] else 8 * _log(rng, 1, 2048)
        elif op == "route":
            c |= {"tokens": _log(rng, 1, 65536)} | _router(rng)
            size = rng.choice([1, 2, 4, 8])  # groups of equal size that hold enough experts for the choice
            if c["experts"] % size == 0 and size > 1:
                c["groups"], c["topk_groups"] = size, rng.randint(1, size)
                c["topk"] = min(c["topk"], c["topk_groups"] * (c["experts"] // size))
            else:
                c["groups"], c["topk_groups"] = 1, 1
            c["bias"] = rng.random() < 0.5
        elif op == "balance":
            c |= {"sequences": _log(rng, 1, 64), "tokens": _log(rng, 1, 4096), "route": rng.random() < 0.5} | _router(rng)
        elif op == "linear4":
            c |= {"rows": _log(rng, 1, 8192), "k": 128 * _log(rng, 1, 64), "n": _log(rng, 1, 8192)}
        else:
            c |= {"experts": _log(rng, 4, 256), "tokens": _log(rng, 1, 8192), "k": 128 * _log(rng, 1, 56), "n": 128 * _log(rng, 1, 16),
                  "skew": rng.choice([0.0, 0.5, 1.0, 1.5]), "mask": rng.choice([0.0, 0.05, 0.3])}
            c["topk"] = rng.randint(1, min(8, c["experts"]))
        w = work(c)
        if op in ("route", "balance") and c["tokens"] * c.get("sequences", 1) * c["experts"] > 1 << 24:
            continue
        if w["flops"] <= 5.7e12 and w["bytes"] <= 8e9:
            return c


def _router(rng):
    c = {"experts": _log(rng, 4, 512), "logits": rng.choice(["fp32", "bf16"]), "scoring": rng.choice(["softmax", "sigmoid"]),
         "normalize": rng.random() < 0.7, "skew": rng.choice([0.0, 0.5, 1.0]), "mask": rng.choice([0.0, 0.05, 0.3])}
    c["topk"] = rng.randint(1, min(16, c["experts"] // 2))
    c["closed"] = rng.choice([0, 0, 1, c["experts"] // 4])
    return c


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"case": c} | {"norm": _prepare_norm, "route": _prepare_router, "balance": _prepare_router, "linear4": _prepare_linear4,
                          "experts4": _prepare_experts4}[c["op"]](c, g)


# ---- the norm ---------------------------------------------------------------------

def _prepare_norm(c, g):
    shape = c["rows"], c["hidden"]
    s = {"x": _normal(shape, g).to(torch.bfloat16), "weight": (1 + 0.1 * _normal(c["hidden"], g)).to(_TYPES[c["weight"]])}
    # a residual stream has grown over the layers, by other amounts in different channels
    s["residual"] = None if c["residual"] == "none" else (_normal(shape, g) * (4 * torch.exp(0.5 * _normal(c["hidden"], g)))).to(_TYPES[c["residual"]])
    if c["grad"]:
        s["dy"] = (1e-3 * _normal(shape, g)).to(torch.bfloat16)
        s["dresidual"] = None if s["residual"] is None else (1e-3 * _normal(shape, g)).to(s["residual"].dtype)
    return s


def _plain_norm(s):
    c, r, w = s["case"], s["residual"], s["weight"].float()
    h = s["x"] if r is None else (s["x"].float() + r.float()).to(r.dtype)
    v = h.float()
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    n = v * rstd * w
    out = {"y": n.to(torch.bfloat16)}
    if r is not None:
        out["residual"] = h
    if c["fp8"]:
        b = n.view(c["rows"], -1, 128)
        sc = b.abs().amax(dim=2) / torch.full_like(b[..., 0], 448.0)
        out["codes"] = torch.where(sc[..., None] > 0, b / sc[..., None], b).to(torch.float8_e4m3fn).view(n.shape)
        out["scales"] = sc
    if c["grad"]:
        dy = s["dy"].float()
        gw = dy * w
        dh = rstd * (gw - v * rstd * rstd * (gw * v).mean(dim=1, keepdim=True))
        if r is not None:
            dh = dh + s["dresidual"].float()
        out["dx"] = dh.to(h.dtype)
        out["dweight"] = (dy * v * rstd).sum(dim=0)
    return out


def _own_norm(s, ep):
    c, r, k = s["case"], s["residual"], s["case"]["hidden"]
    got = ep.rms_norm(s["x"], s["weight"], EPS, residual=r, fp8=c["fp8"])
    out = {"y": got["y"]}
    if r is not None:
        out["residual"] = got["residual"]
    if c["fp8"]:
        codes, out["scales"] = ep.fp8_row_views(got["rows"], k)
        out["codes"] = codes.view(torch.float8_e4m3fn)
    if c["grad"]:
        out["dx"], out["dweight"] = ep.rms_norm_backward(s["dy"], s["x"] if r is None else got["residual"], s["weight"], EPS,
                                                         dresidual=s["dresidual"])
    return out


def _exact_norm(s):
    c, r, w = s["case"], s["residual"], s["weight"].double()
    total = s["x"].double() if r is None else s["x"].double() + r.double()
    h = total if r is None else total.to(r.dtype).double()  # the norm is taken of what is written
    scale = 1 / torch.sqrt(torch.einsum("tc,tc->t", h, h) / c["hidden"] + EPS)
    n = torch.einsum("tc,t,c->tc", h, scale, w)
    out = {"y": n}
    if r is not None:
        out["residual"] = total
    if c["fp8"]:
        a = n.abs().unflatten(1, (-1, 128)).max(dim=2).values / 448
        out["codes"], out["scales"] = n / a.clamp(min=1e-300).repeat_interleave(128, 1), a
    if c["grad"]:
        d = s["dy"].double()
        inner = torch.einsum("tc,c,tc->t", d, w, h) / c["hidden"]
        dh = scale[:, None] * d * w - h * (scale ** 3 * inner)[:, None]
        out["dx"] = dh if r is None else dh + s["dresidual"].double()
        out["dweight"] = torch.einsum("tc,tc,t->c", d, h, scale)
    return out


# ---- the router -------------------------------------------------------------------

def _prepare_router(c, g):
    lead = (c["sequences"], c["tokens"]) if c["op"] == "balance" else (c["tokens"],)
    logits = _normal((*lead, c["experts"]), g) + c["skew"] * _normal(c["experts"], g)
    if c["closed"]:  # experts taken out of service, leaving enough for the choice or not
        logits[..., torch.randperm(c["experts"], generator=g, device="cuda")[:c["closed"]]] = -math.inf
    s = {"logits": logits.to(_TYPES[c["logits"]])}
    s["mask"] = torch.rand(lead, generator=g, device="cuda") >= c["mask"] if c["mask"] else None  # False: a padded token
    if c["op"] == "route":
        s["bias"] = 0.2 * _normal(c["experts"], g) if c["bias"] else None
    else:
        idx = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[..., :c["topk"]]
        open_ = torch.gather(s["logits"], -1, idx) > -math.inf
        s["topk_idx"] = torch.where(open_ if s["mask"] is None else open_ & s["mask"][..., None], idx, -1)
        s["dweights"] = 1e-3 * _normal((*lead, c["topk"]), g)
        s["dloss"] = torch.ones(1, device="cuda")
    return s


def _plain_choice(logits, c, bias, mask):
    key = logits.float() if bias is None else logits.float() + bias
    if c.get("groups", 1) > 1:
        members = key.unflatten(-1, (c["groups"], -1))
        best = torch.sort(members, dim=-1, descending=True).values[..., :2].sum(dim=-1)
        order = torch.sort(best, dim=-1, descending=True, stable=True).indices[..., :c["topk_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(-1, order, True)
        key = torch.where(kept[..., None], members, -math.inf).view(key.shape)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :c["topk"]]
    fine = torch.gather(key, -1, idx) != -math.inf
    return torch.where(fine if mask is None else fine & mask[..., None], idx, -1)


def _scores(logits, c):
    """(softmax, or sigmoid; its sum over the experts)."""
    v = logits.float()
    if c["scoring"] == "sigmoid":
        p = 1 / (1 + torch.exp(-v))
        return p, p.sum(dim=-1, keepdim=True)
    e = torch.exp(v - v.amax(dim=-1, keepdim=True))
    e = e / e.sum(dim=-1, keepdim=True)
    return e, None


def _plain_weights(logits, idx, c):
    """The chosen experts' scores, and by what they are divided."""
    chosen = idx >= 0
    if c["scoring"] == "softmax" and c["normalize"]:
        v = torch.where(chosen, torch.gather(logits.float(), -1, idx.clamp(min=0)), -math.inf)
        e = torch.where(chosen, torch.exp(v - v.amax(dim=-1, keepdim=True)), 0.0)
        return e, torch.where(chosen.any(dim=-1, keepdim=True), e.sum(dim=-1, keepdim=True), 1.0)
    p = torch.where(chosen, torch.gather(_scores(logits, c)[0], -1, idx.clamp(min=0)), 0.0)
    return p, p.sum(dim=-1, keepdim=True) + 1e-20 if c["normalize"] else torch.ones_like(p[..., :1])


def _plain_balance(logits, idx, c):
    """(loss, counts, factors F): loss = sum F p."""
    S, E = idx.shape[0], c["experts"]
    counts = torch.zeros(S, E + 1, dtype=torch.int32, device="cuda")
    counts.scatter_add_(1, torch.where(idx >= 0, idx, E).view(S, -1), torch.ones_like(idx, dtype=torch.int32).view(S, -1))
    counts = counts[:, :E]
    used = (idx >= 0).any(dim=-1)
    pairs, tokens = counts.sum(dim=1, keepdim=True).float(), used.sum(dim=1, keepdim=True).float()
    factors = COEF * E / S * counts / (pairs * tokens).clamp(min=1.0)
    p, total = _scores(logits, c)
    p = torch.where(used[..., None], p if total is None else p / total, 0.0)
    return (factors * p.double().sum(dim=1).float()).sum().view(1), counts, factors


def _plain_router_grad(logits, idx, c, dweights, factors, dloss):
    p, total = _scores(logits, c)
    used = (idx >= 0).any(dim=-1, keepdim=True)
    q = p if total is None else p / total
    f = factors[:, None, :]  # nearly equal where the load is balanced: its differences from the mean in 64 bits
    inner = (f.double() - (f.double() * q).sum(dim=-1, keepdim=True) / q.double().sum(dim=-1, keepdim=True)).float()
    d = dloss * (q * inner if total is None else inner / total * p * (1 - p))
    d = torch.where(used, d, 0.0)
    if dweights is not None:
        w, by = _plain_weights(logits, idx, c)
        w, g = w / by, torch.where(idx >= 0, dweights, 0.0)
        if c["scoring"] == "softmax":
            inner = (g * w).sum(dim=-1, keepdim=True)
            at = w * (g - inner) if c["normalize"] else w * g
            if not c["normalize"]:
                d = d - p * inner
        else:
            s = torch.where(idx >= 0, torch.gather(p, -1, idx.clamp(min=0)), 0.0)
            at = s * (1 - s) * ((g - (g * w).sum(dim=-1, keepdim=True)) / by if c["normalize"] else g)
        more = torch.zeros(*d.shape[:-1], d.shape[-1] + 1, device="cuda").scatter_add_(-1, torch.where(idx >= 0, idx, d.shape[-1]), at)
        d = d + more[..., :-1]
    return d.to(logits.dtype)


def _plain_router(s):
    c, logits = s["case"], s["logits"]
    if c["op"] == "route":
        idx = _plain_choice(logits, c, s["bias"], s["mask"])
        w, by = _plain_weights(logits, idx, c)
        return {"idx": idx, "weights": w / by}
    out = {}
    idx = s["topk_idx"]
    if c["route"]:
        idx = out["idx"] = _plain_choice(logits, c, None, s["mask"])
        w, by = _plain_weights(logits, idx, c)
        out["weights"] = w / by
    out["loss"], out["counts"], factors = _plain_balance(logits, idx, c)
    out["dlogits"] = _plain_router_grad(logits, idx, c, s["dweights"] if c["route"] else None, factors, s["dloss"])
    return out


def _own_router(s, ep):
    c, logits = s["case"], s["logits"]
    how = {"scoring": c["scoring"], "normalize": c["normalize"]}
    if c["op"] == "route":
        idx, weights = ep.route(logits, c["topk"], bias=s["bias"], mask=s["mask"], groups=c["groups"], topk_groups=c["topk_groups"], **how)
        return {"idx": idx, "weights": weights}
    out = {}
    idx = s["topk_idx"]
    if c["route"]:
        idx, out["weights"] = ep.route(logits, c["topk"], mask=s["mask"], **how)
        out["idx"] = idx
    got = ep.balance_loss(logits, idx, COEF, scoring=c["scoring"])
    out["loss"], out["counts"] = got["loss"], got["counts"]
    out["dlogits"] = ep.router_backward(logits, idx, s["dweights"] if c["route"] else None, factors=got["factors"], dloss=s["dloss"], **how)
    return out


def _exact_router(s):
    c = s["case"]
    lead, E, K = s["logits"].shape[:-1], c["experts"], c["topk"]
    v = s["logits"].double().view(-1, E)
    if c["op"] == "route" or c["route"]:  # the operator's keys are rounded to 32 bits once
        key = v if s.get("bias") is None else v + s["bias"].double()
        key = key.float()
        groups = c.get("groups", 1)
        if groups > 1:
            two = torch.topk(key.view(len(key), groups, -1), min(2, E // groups), dim=-1).values
            best = (two.double().sum(dim=-1)).float()
            rank = torch.argsort(-best, dim=1, stable=True)[:, :c["topk_groups"]]
            keep = (rank[:, :, None] == torch.arange(groups, device="cuda")).any(dim=1)
            key = key.masked_fill(~keep.repeat_interleave(E // groups, dim=1), -math.inf)
        idx = torch.argsort(-key, dim=1, stable=True)[:, :K]
        idx = idx.masked_fill(key.gather(1, idx) == -math.inf, -1)
        if s["mask"] is not None:
            idx = idx.masked_fill(~s["mask"].view(-1, 1), -1)
    else:
        idx = s["topk_idx"].view(-1, K)
    chosen = idx >= 0
    at = idx.clamp(min=0)
    if c["scoring"] == "softmax":
        score = torch.exp(v - torch.logsumexp(v, dim=1, keepdim=True)).nan_to_num(0.0)
        share, slope = score, None
        picked = torch.where(chosen, score.gather(1, at), 0.0)
        if c["normalize"]:
            lv = torch.where(chosen, v.gather(1, at), -math.inf)
            picked = torch.exp(lv - torch.logsumexp(lv, dim=1, keepdim=True)).nan_to_num(0.0)
    else:
        score = torch.sigmoid(v)
        total = score.sum(dim=1, keepdim=True)
        share = score / total.clamp(min=1e-300)
        slope = score * torch.sigmoid(-v)
        picked = torch.where(chosen, score.gather(1, at), 0.0)
        by = picked.sum(dim=1, keepdim=True) + 1e-20
        if c["normalize"]:
            picked = picked / by
    if c["op"] == "route":
        return {"idx": idx.view(*lead, K), "weights": picked.view(*lead, K)}
    out = {}
    if c["route"]:
        out["idx"], out["weights"] = idx.view(*lead, K), picked.view(*lead, K)
    S, T = lead
    used = chosen.any(dim=1)
    counts = torch.stack([torch.bincount(row[row >= 0], minlength=E) for row in idx.view(S, -1)])
    pairs = counts.sum(dim=1).double().clamp(min=1)
    tokens = used.view(S, T).sum(dim=1).double().clamp(min=1)
    factors = COEF * E * counts.double() / (S * pairs * tokens)[:, None]
    mass = torch.einsum("ste,st->se", share.view(S, T, E), used.view(S, T).double())
    out["loss"], out["counts"] = (factors * mass).sum().view(1), counts.to(torch.int32)
    f = factors.repeat_interleave(T, dim=0)
    inner = f - torch.einsum("te,te->t", f, share)[:, None]
    d = (share * inner if slope is None else slope * inner / total) * used[:, None] * s["dloss"].double()
    if c["route"]:
        g = torch.where(chosen, s["dweights"].double().view(-1, K), 0.0)
        mean = torch.einsum("tk,tk->t", g, picked)[:, None]
        if c["scoring"] == "softmax":
            near = picked * (g - mean) if c["normalize"] else picked * g
            if not c["normalize"]:
                d = d - share * mean
        else:
            near = torch.where(chosen, slope.gather(1, at), 0.0) * ((g - mean) / by if c["normalize"] else g)
        d = d.scatter_add(1, at, torch.where(chosen, near, 0.0))
    out["dlogits"] = d.view(*lead, E)
    return out


# ---- 4-bit experts ----------------------------------------------------------------

def _mxfp4(v):
    """(e2m1 values, exponents) of fp32 rows [..][K]: one exponent per 32 channels, values rounded to nearest even."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(dim=-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    a = torch.ldexp(b, -e).clamp(-6, 6)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    return torch.round(a / step) * step, e


def _codes(values, e):
    """What memory holds of them: packed codes [..][K/2] and exponents [..][K/32]."""
    a = values.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(values).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8).squeeze(-1)


def _values4(codes, e):
    """The fp32 values of packed codes and exponents."""
    t = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    t = torch.cat([t, -t])
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], dim=-1).flatten(-2)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (e.int() - 127)[..., None]).flatten(-2)


def _weight4(experts, n, k, g):
    codes = torch.empty(experts, n, k // 2, dtype=torch.uint8, device="cuda")
    e = torch.empty(experts, n, k // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for i in range(0, experts, step):
        m = min(step, experts - i)
        codes[i:i + m], e[i:i + m] = _codes(*_mxfp4(_normal((m, n, k), g) * k ** -0.5))
    return codes, e


def _prepare_linear4(c, g):
    s = {"x": _normal((c["rows"], c["k"]), g).to(torch.bfloat16)}
    w, e = _weight4(1, c["n"], c["k"], g)
    s["w"], s["w_scales"] = w[0], e[0]
    return s


def _prepare_experts4(c, g):
    logits = _normal((c["tokens"], c["experts"]), g) + c["skew"] * _normal((c["experts"],), g)
    idx = torch.topk(logits, c["topk"], dim=1).indices
    keep = torch.rand(idx.shape, generator=g, device="cuda") >= c["mask"]
    keep[0, 0] = True
    counts = torch.bincount(idx[keep], minlength=c["experts"]).to(torch.int32)
    rows = c["tokens"] * c["topk"]  # the worst case, whatever is masked; rows past the groups unused
    s = {"counts": counts, "offsets": (torch.cumsum(counts, 0) - counts).to(torch.int32), "host_counts": counts.tolist()}
    s["x"], s["x_scales"] = _codes(*_mxfp4(_normal((rows, c["k"]), g)))
    s["w13"], s["w13_scales"] = _weight4(c["experts"], 2 * c["n"], c["k"], g)
    s["w2"], s["w2_scales"] = _weight4(c["experts"], c["k"], c["n"], g)
    # the buffer that a serving loop keeps; rows of no expert stay zero
    s["out"] = torch.zeros(rows, c["k"], dtype=torch.bfloat16, device="cuda")
    return s


def _plain_linear4(s):
    v, e = _mxfp4(s["x"].float())
    return (torch.ldexp(v, e).flatten(-2) @ _values4(s["w"], s["w_scales"]).t()).to(torch.bfloat16)


def _plain_experts4(s):
    n, lo = s["case"]["n"], 0
    for i, m in enumerate(s["host_counts"]):  # ragged groups: their products one by one
        if m:
            y = _values4(s["x"][lo:lo + m], s["x_scales"][lo:lo + m]) @ _values4(s["w13"][i], s["w13_scales"][i]).t()
            gate, up = y[:, :n], y[:, n:]
            v, e = _mxfp4(gate * torch.sigmoid(gate) * up)
            s["out"][lo:lo + m] = (torch.ldexp(v, e).flatten(-2) @ _values4(s["w2"][i], s["w2_scales"][i]).t()).to(torch.bfloat16)
        lo += m
    return s["out"]


def _own_linear4(s, ep):
    codes, scales = ep.quantize_fp4(s["x"])
    return ep.expert_gemm_fp4(codes, scales, s["w"], s["w_scales"])


def _own_experts4(s, ep):
    rows = {"counts": s["counts"], "offsets": s["offsets"]}
    h, hs = ep.expert_swiglu_fp4(s["x"], s["x_scales"], s["w13"], s["w13_scales"], **rows)
    return ep.expert_gemm_fp4(h, hs, s["w2"], s["w2_scales"], out=s["out"], **rows)


def _matrix64(codes, e):
    """The 64-bit values of MXFP4 rows, from the formats' definitions."""
    t = []
    for b in range(16):
        x, m = (b >> 1) & 3, b & 1
        v = m * 0.5 if x == 0 else (1 + m / 2) * 2.0 ** (x - 1)
        t.append(-v if b & 8 else v)
    t = torch.tensor(t, dtype=torch.float64, device="cuda")
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    out[..., 0::2], out[..., 1::2] = t[(codes % 16).int()], t[(codes // 16).int()]
    return out * _power64(e.int() - 127).repeat_interleave(32, -1)


def _power64(e):
    """2^e, put together from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest64(v):
    """MXFP4 of 64-bit rows as 64-bit values: for each the nearest of the eight magnitudes, ties to the even code."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().max(dim=-1, keepdim=True).values
    unit = _power64(((top.view(torch.int64) >> 52) - 1025).clamp(-127, 127))  # the exponent's bits, less 1023 and 2
    a = (b / unit).abs()
    edges = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    q = torch.zeros_like(a)
    for i, edge in enumerate(edges):  # a tie goes up where the code above is even
        q = torch.where(a >= edge if (i + 1) % 2 == 0 else a > edge, grid[i + 1], q)
    return (torch.copysign(q, b) * unit).flatten(-2)


def _exact_linear4(s):
    return torch.einsum("rk,nk->rn", _nearest64(s["x"].double()), _matrix64(s["w"], s["w_scales"]))


def _exact_experts4(s):
    n = s["case"]["n"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    ends = torch.tensor(s["host_counts"]).cumsum(0).tolist()
    for i, (m, end) in enumerate(zip(s["host_counts"], ends)):
        if m:
            rows = slice(end - m, end)
            y = torch.einsum("rk,nk->rn", _matrix64(s["x"][rows], s["x_scales"][rows]), _matrix64(s["w13"][i], s["w13_scales"][i]))
            h = y[:, :n] / (1 + torch.exp(-y[:, :n])) * y[:, n:]
            out[rows] = torch.einsum("rk,nk->rn", _nearest64(h), _matrix64(s["w2"][i], s["w2_scales"][i]))
    return out


# ---- one pass ---------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "route": _plain_router, "balance": _plain_router, "linear4": _plain_linear4,
                "experts4": _plain_experts4}[op](state)
    import combine_get_dispatch_histograms_gb300 as ep
    return {"norm": _own_norm, "route": _own_router, "balance": _own_router, "linear4": _own_linear4,
            "experts4": _own_experts4}[op](state, ep)


def work(case):
    c = case
    if c["op"] == "norm":
        n, r = c["rows"] * c["hidden"], {"none": 0, "bf16": 2, "fp32": 4}[c["residual"]]
        b, f = n * (4 + 2 * r + (33 / 32 if c["fp8"] else 0)) + c["hidden"] * 4, 8.0 * n
        if c["grad"]:  # dy, h and its gradient read, a gradient written
            b, f = b + n * (2 + (3 * r if r else 4)) + c["hidden"] * 8, f + 12.0 * n
        return {"bytes": float(b), "flops": f}
    if c["op"] in ("route", "balance"):
        tokens = c["tokens"] * c.get("sequences", 1)
        n, e = tokens * c["experts"], 2 if c["logits"] == "bf16" else 4
        if c["op"] == "route":
            return {"bytes": float(n * e + tokens * c["topk"] * 12), "flops": 8.0 * n}
        b = 2 * n * e + tokens * c["topk"] * 8 + c["sequences"] * c["experts"] * 4  # logits read, their gradient written
        return {"bytes": float(b + (tokens * c["topk"] * 8 if c["route"] else 0)), "flops": 20.0 * n}
    per = 0.5 + 1 / 32
    if c["op"] == "linear4":
        m, k, n = c["rows"], c["k"], c["n"]
        return {"bytes": m * (2.0 * k + 2 * n) + n * k * per, "flops": 2.0 * m * n * k}
    pairs = c["tokens"] * c["topk"] * (1.0 - c["mask"])
    hit = c["experts"] * (1.0 - (1.0 - c["topk"] * (1.0 - c["mask"]) / c["experts"]) ** c["tokens"])
    return {"bytes": pairs * (c["k"] * per + 2 * c["k"]) + max(1.0, hit) * 3 * c["n"] * c["k"] * per,
            "flops": 6.0 * pairs * c["n"] * c["k"]}


def exact(case, seed):
    c = dict(case)
    if work(c)["flops"] > 1.4e13:
        return None
    s = prepare(c, seed)
    return {"norm": _exact_norm, "route": _exact_router, "balance": _exact_router, "linear4": _exact_linear4,
            "experts4": _exact_experts4}[c["op"]](s)
