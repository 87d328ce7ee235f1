"""The router of a mixture of experts, the group and the experts' product on 8-bit floating-point
weights with a scale for each block of 128 x 128, and the layer norm in front of them, as measured
workloads: their cases, inputs, plain forms, calls and exact results.

fp8        per token t and group g of 128 inputs s[t, g] = max |x| / 448, c = e4m3(x (448 / max |x|)), fp32;
           y_i[t, o] = sum_g s[t, g] S_i[o / 128, g] sum_{k in g} c[t, k] q_i[o, k] + (X B^T) A_i^T
experts    the same for rows listed by expert, each with its expert's weights, B (or one B for all) and A
route      scores s = softmax(l) or sigmoid(l) over a token's experts; experts of logit -inf are out.
           The order of choice is that of s + bias (of l without a bias; equal values: the lower expert),
           first over groups of experts (by their best value or the sum of their two best), then over the
           experts of the groups that stay.  ids of the top_k, -1 where experts run out;
           weights scale s, or scale s / sum of the chosen s
           backward: d_l for d_weights, the ids held
norm       mean and 1 / sqrt(variance + eps) of a row, y = (x - mean) rstd w + b
           backward: dx, dw = sum_t dy xhat, db = sum_t dy (fp32)

With `own` false run() computes the plain forms in elementary torch operations; with `own` true it
calls the library.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# --------------------------------------------------------------------------- cases
def _named(c, name):
    return {"name": name, **c} if name else c


def _fp8(T, d, rows, r, name=None):
    return _named({"op": "fp8", "T": T, "d": d, "rows": ",".join(str(n) for n in rows), "r": r}, name)


def _experts(T, k, n_exp, d, rows, r, share, drop, name=None):
    return _named({"op": "experts", "T": T, "k": k, "n_exp": n_exp, "d": d, "rows": ",".join(str(n) for n in rows), "r": r,
                   "share": share, "drop": drop}, name)


def _route(back, T, n_exp, k, score, bias, groups, keep, best, renorm, dtype, masked, name=None):
    return _named({"op": "route", "back": back, "T": T, "n_exp": n_exp, "k": k, "score": score, "bias": bias,
                   "groups": groups, "keep": keep, "best": best, "renorm": renorm, "dtype": dtype, "masked": masked}, name)


def _norm(back, T, d, dtype, name=None):
    return _named({"op": "norm", "back": back, "T": T, "d": d, "dtype": dtype}, name)


def listed():
    return [
        # one generated token through the Q/K/V group of an 8B decoder (grouped-query heads)
        _fp8(1, 4096, (4096, 1024, 1024), 64, "fp8_qkv_t1"),
        # a ragged batch of requests through the long-row down projection
        _fp8(77, 14336, (4096,), 64, "fp8_down_t77"),
        # a 2048-token prompt through gate/up
        _fp8(2048, 4096, (11008, 11008), 64, "fp8_gateup_t2048"),
        # one generated token's four routed rows through the experts' gate/up, one B for all experts
        _experts(1, 4, 60, 2048, (1408, 1408), 64, "all", 0, "experts_gateup_t1"),
        # a prompt of odd length through them, a B for each expert, one pair in 16 without an expert
        _experts(4095, 4, 60, 2048, (1408, 1408), 64, "expert", 16, "experts_gateup_t4095"),
        # the choice of one generated token (latency)
        _route(False, 1, 60, 4, "softmax", False, 1, 1, 1, True, "f16", False, "route_t1"),
        # a large prompt batch over 256 experts in 8 groups of which 4 stay, a bias for balance, padded tokens
        _route(False, 32767, 256, 8, "sigmoid", True, 8, 4, 2, True, "f32", True, "route_t32767_groups"),
        # the router's gradient at a training batch, plain softmax scores (every logit of a token has one)
        _route(True, 16384, 60, 4, "softmax", False, 1, 1, 1, False, "f32", False, "route_back_t16384"),
        # the norm of one generated token (latency)
        _norm(False, 1, 4096, "f16", "norm_t1"),
        # the norm of a large prompt batch
        _norm(False, 16383, 4096, "f16", "norm_t16383"),
        # its gradients at a small batch in 32 bits, odd length
        _norm(True, 515, 2048, "f32", "norm_back_t515_f32"),
        # its gradients at a training batch
        _norm(True, 16384, 4096, "f16", "norm_back_t16384"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp8", "fp8", "experts", "experts", "route", "route", "norm"])
    ranks = [0, 8, 24, 64, 128, 256]
    if op == "fp8":
        while True:
            T, d = _spread(rng, 1, 4096), 128 * _spread(rng, 1, 112)
            rows = tuple(_spread(rng, 1, 16384) for _ in range(rng.randint(1, 3)))
            if T * d * sum(rows) <= 2048 * 4096 * 22016:
                return _fp8(T, d, rows, rng.choice(ranks))
    if op == "experts":
        while True:
            T, n_exp, d = _spread(rng, 1, 8192), _spread(rng, 2, 128), 128 * _spread(rng, 1, 32)
            k = rng.randint(1, min(8, n_exp))
            rows = tuple(_spread(rng, 1, 2816) for _ in range(rng.randint(1, 2)))
            if T * k * d * sum(rows) <= 4095 * 4 * 2048 * 2816 and n_exp * d * sum(rows) <= 60 * 2048 * 2816 and T * d <= 4095 * 2048:
                return _experts(T, k, n_exp, d, rows, rng.choice(ranks[:5]), rng.choice(["all", "expert"]), rng.choice([0, 0, 4, 16]))
    back = rng.random() < 0.4
    dtype = rng.choice(["f16", "f32"])
    if op == "norm":
        while True:
            T, d = _spread(rng, 1, 65536), _spread(rng, 16, 16384)
            if T * d * (2 if dtype == "f32" else 1) <= 16384 * 4096:
                return _norm(back, T, d, dtype)
    n_exp = _spread(rng, 2, 256)
    T = _spread(rng, 1, 32767 * 256 // n_exp)
    groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if n_exp % g == 0])
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(8, n_exp // groups * keep))
    bias = rng.random() < 0.5
    renorm = rng.random() < 0.6 and not (back and k == 1)  # one renormalised weight is a constant
    return _route(back, T, n_exp, k, rng.choice(["softmax", "sigmoid"]), bias, groups, keep, rng.choice([1, 2]),
                  renorm, dtype, rng.random() < 0.4)


def _rows(case):
    return [int(n) for n in case["rows"].split(",")]


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    op, T = case["op"], case["T"]
    if op == "fp8":
        d, r, n = case["d"], case["r"], sum(_rows(case))
        return {"bytes": 2 * T * d + n * d + n * d // 4096 + 2 * r * (d + n) + 2 * T * n,
                "flops": 2 * T * n * d + 2 * r * T * (d + n)}
    if op == "experts":
        k, E, d, r, n = case["k"], case["n_exp"], case["d"], case["r"], sum(_rows(case))
        pairs = T * k - (T * k // case["drop"] if case["drop"] else 0)
        used = min(E, max(pairs, 1))  # experts that have rows, at most
        b = (used if case["share"] == "expert" else 1) * r * d
        return {"bytes": 2 * T * d + used * (n * d + n * d // 4096 + 2 * r * n) + 2 * b + 2 * pairs * n + 4 * (pairs + E + 1),
                "flops": 2 * pairs * n * d + 2 * r * (pairs * n + (pairs if case["share"] == "expert" else T) * d)}
    e = 2 if case["dtype"] == "f16" else 4
    if op == "route":
        E, k = case["n_exp"], case["k"]
        return {"bytes": T * E * e * (2 if case["back"] else 1) + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 5 * T * E}
    n = T * case["d"]
    return {"bytes": (3 if case["back"] else 2) * n * e + 2 * case["d"] * e + 8 * T, "flops": (11 if case["back"] else 8) * n}


# --------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, T, d):
    """Rows with a power-law channel spectrum."""
    chan = torch.arange(1, d + 1, device="cuda").float() ** -0.5
    chan = (chan * math.sqrt(d) / chan.norm())[torch.randperm(d, generator=gen, device="cuda")]
    return (_randn(gen, T, d) * chan).half()


def _blocks(w):
    """Codes and 128 x 128 scales of w [..., n, d] (d a multiple of 128)."""
    *e, n, d = w.shape
    pad = torch.zeros(*e, -(-n // 128) * 128, d, device=w.device)
    pad[..., :n, :] = w
    v = pad.view(*e, -(-n // 128), 128, d // 128, 128)
    s = v.abs().amax((-3, -1)).clamp(min=1e-12) / 448.0
    q = (v / s[..., :, None, :, None]).to(E4M3).view(*e, -1, d)[..., :n, :].contiguous()
    return q, s.contiguous()


def _weights(gen, *shape):
    """Weights with a few outlier input columns."""
    w = 0.02 * _randn(gen, *shape)
    w[..., : min(4, shape[-1])] *= 10.0
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op, T = case["op"], case["T"]
    if op == "fp8":
        d, r = case["d"], case["r"]
        s["x"] = _activations(gen, T, d)
        s["q"], s["scale"] = [list(v) for v in zip(*[_blocks(_weights(gen, n, d)) for n in _rows(case)])]
        s["a"] = [(_randn(gen, n, r) * (0.02 * 0.03 * math.sqrt(d / max(r, 1)))).half() for n in _rows(case)]
        s["b"] = (_randn(gen, r, d) / math.sqrt(d)).half()
    elif op == "experts":
        k, E, d, r = case["k"], case["n_exp"], case["d"], case["r"]
        s["x"] = _activations(gen, T, d)
        # distinct experts per token from scores with a per-expert bias (some experts are busier)
        ids = torch.topk(_randn(gen, T, E) + 0.7 * _randn(gen, 1, E), k, dim=1).indices.reshape(-1)
        if case["drop"]:
            ids[torch.randperm(T * k, generator=gen, device="cuda")[: T * k // case["drop"]]] = E
        key, order = torch.sort(ids, stable=True)
        offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
        s["n_rows"] = int(offsets[-1])
        s["longest"] = int((offsets[1:] - offsets[:-1]).max())
        s["offsets"], s["token"] = offsets, (order // k)[: s["n_rows"]].to(torch.int32)
        s["q"], s["scale"] = [list(v) for v in zip(*[_blocks(_weights(gen, E, n, d)) for n in _rows(case)])]
        s["a"] = [(_randn(gen, E, n, r) * (0.02 * 0.03 * math.sqrt(d / max(r, 1)))).half() for n in _rows(case)]
        s["b"] = (_randn(gen, *((E,) if case["share"] == "expert" else ()), r, d) / math.sqrt(d)).half()
    elif op == "route":
        E, t = case["n_exp"], DTYPES[case["dtype"]]
        s["logits"] = (1.5 * _randn(gen, T, E) + 0.7 * _randn(gen, 1, E)).to(t)
        if case["masked"]:  # one token in 16 is padding, one logit in 32 is masked
            s["logits"][torch.rand(T, E, generator=gen, device="cuda") < 1 / 32] = -math.inf
            s["logits"][torch.rand(T, generator=gen, device="cuda") < 1 / 16] = -math.inf
        s["bias"] = 0.1 * _randn(gen, E) if case["bias"] else None
        if case["back"]:
            s["ids"] = _plain_route(s)[0]
            s["dw"] = _randn(gen, T, case["k"])
    else:
        d, t = case["d"], DTYPES[case["dtype"]]
        s["x"] = (_randn(gen, T, d) * (0.3 + torch.rand(1, d, generator=gen, device="cuda")) + 0.5 * _randn(gen, T, 1)).to(t)
        s["w"], s["bias"] = (1.0 + 0.2 * _randn(gen, d)).to(t), (0.1 * _randn(gen, d)).to(t)
        if case["back"]:
            s["dy"] = _randn(gen, T, d).to(t)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
    if own:
        s["plan"] = _plan(s)
    return s


EPS = 1e-5
SCALE = 2.5  # of the router's weights


# --------------------------------------------------------------------------- the library's calls
def _plan(s):
    """What a program keeps between calls: weights in the device layout, a workspace."""
    from rank_error_compensation_amd import glowq as g
    c = s["case"]
    T = c["T"]
    empty = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    if c["op"] == "fp8":
        return g, [g.QWeight.from_fp8(q, sc) for q, sc in zip(s["q"], s["scale"])], empty(g.fp8_workspace_bytes(T, c["d"], c["r"]))
    if c["op"] == "experts":
        mods = [g.MoeModule.stack([g.QWeight.from_fp8(q[e], sc[e]) for e in range(c["n_exp"])], a)
                for q, sc, a in zip(s["q"], s["scale"], s["a"])]
        share = g.MOE_SHARE_EXPERT if c["share"] == "expert" else g.MOE_SHARE_ALL
        return g, (mods, share), g.init_workspace(empty(g.moe_fp8_workspace_bytes(s["n_rows"], T, c["d"], c["r"], share)))
    if c["op"] == "route":
        return g, None, g.init_workspace(empty(8192))
    return g, None, empty(g.layer_norm_workspace_bytes(T, c["d"])) if c["back"] else None


def _run_own(s):
    c = s["case"]
    g, kept, ws = s["plan"]
    if c["op"] == "fp8":
        r = c["r"]
        return g.group_forward_fp8(s["x"], kept, s["b"] if r else None, s["a"] if r else [], r, r > 0, workspace=ws)
    if c["op"] == "experts":
        r = c["r"]
        mods, share = kept
        return g.moe_forward_fp8(s["x"], c["n_exp"], mods, s["b"] if r else None, share, r, r > 0, s["token"], s["offsets"],
                                 s["n_rows"], workspace=ws)
    if c["op"] == "route":
        if c["back"]:
            return g.moe_route_backward(s["dw"], s["logits"], s["ids"], score=c["score"], renorm=c["renorm"], scale=SCALE, workspace=ws)
        return g.moe_route(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_group=c["groups"], keep_groups=c["keep"],
                           group_best=c["best"], renorm=c["renorm"], scale=SCALE, workspace=ws)
    if c["back"]:
        return g.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], workspace=ws)
    return g.layer_norm(s["x"], s["w"], s["bias"], EPS)


# --------------------------------------------------------------------------- plain forms
def _dequant(q, scale):
    """fp32 [..., n, d] of codes and their 128 x 128 scales."""
    full = scale.repeat_interleave(128, -2)[..., : q.shape[-2], :].repeat_interleave(128, -1)
    return q.float() * full


def _plain_codes(x):
    """What the codes of x stand for, fp32."""
    v = x.float().view(x.shape[0], -1, 128)
    top = v.abs().amax(2, keepdim=True)
    most = torch.full_like(top, 448.0)  # two tensors: a quotient with a number is a product with an inverse
    inv = torch.where(top > 0, most / top, torch.zeros_like(top))
    return ((v * inv).to(E4M3).float() * (top / most)).view(x.shape)


def _plain_fp8(s):
    x = _plain_codes(s["x"])
    proj = s["x"].float() @ s["b"].float().t()
    return [(x @ _dequant(q, sc).t() + proj @ a.float().t()).half() for q, sc, a in zip(s["q"], s["scale"], s["a"])]


def _plain_experts(s):
    c = s["case"]
    E, n, cap = c["n_exp"], s["n_rows"], s["longest"]
    row = torch.arange(n, device="cuda")
    expert = torch.searchsorted(s["offsets"].long(), row, right=True) - 1
    place = row - s["offsets"].long()[expert]
    x, xh = _plain_codes(s["x"])[s["token"].long()], s["x"].float()[s["token"].long()]

    def product(rows, w):  # rows [n][d] times the experts' w [E][o][d]
        if n <= E:
            return (w[expert].float() * rows[:, None]).sum(2)
        padded = torch.zeros(E, rows.shape[1], cap, device="cuda")
        padded[expert, :, place] = rows
        return torch.bmm(w.float(), padded)[expert, :, place]

    proj = product(xh, s["b"]) if c["share"] == "expert" else xh @ s["b"].float().t()
    if n <= E:
        return [((_dequant(q[expert], sc[expert]) * x[:, None]).sum(2) + product(proj, a)).half()
                for q, sc, a in zip(s["q"], s["scale"], s["a"])]
    return [(product(x, _dequant(q, sc)) + product(proj, a)).half() for q, sc, a in zip(s["q"], s["scale"], s["a"])]


def _plain_scores(s, logits):
    if s["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True).clamp(min=-1e30))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(s):
    """In 64 bits: values next to one another have to be told apart."""
    c = s["case"]
    T, E, k, G = c["T"], c["n_exp"], c["k"], c["groups"]
    logits = s["logits"].double()
    out = logits == -math.inf
    score = _plain_scores(s, logits)
    value = logits if s["bias"] is None else (score + s["bias"].double()).masked_fill(out, -math.inf)
    if G > 1:
        # a group's standing: its best value, or the sum of its two best scores (with the bias)
        by = value if c["best"] == 1 else (score + (0.0 if s["bias"] is None else s["bias"].double())).masked_fill(out, -math.inf)
        best = torch.sort(by.view(T, G, E // G), dim=2, descending=True).values[:, :, : c["best"]]
        stand = torch.where(best[:, :, 0] == -math.inf, best[:, :, 0], best.masked_fill(best == -math.inf, 0.0).sum(2))
        order = torch.sort(stand, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        value = value.masked_fill(~stays.repeat_interleave(E // G, 1), -math.inf)
    top = torch.sort(value, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k].masked_fill(top.values[:, :k] == -math.inf, -1)
    return ids.to(torch.int32), _plain_weights(s, logits, score, ids).float()


def _plain_weights(s, logits, score, ids):
    chosen = score.gather(1, ids.clamp(min=0).long()).masked_fill(ids < 0, 0.0)
    if s["case"]["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    return SCALE * chosen


def _plain_route_back(s):
    logits, ids = s["logits"].float(), s["ids"].long()
    score = _plain_scores(s, logits)
    live = ids >= 0
    chosen = score.gather(1, ids.clamp(min=0)).masked_fill(~live, 0.0)
    d = (SCALE * s["dw"]).masked_fill(~live, 0.0)
    if s["case"]["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-30)
        d = (d - (d * chosen).sum(1, keepdim=True) / total) / total
        d = d.masked_fill(~live, 0.0)
    d_score = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), d)
    if s["case"]["score"] == "sigmoid":
        d_logits = d_score * score * (1.0 - score)
    else:
        d_logits = score * (d_score - (d_score * score).sum(1, keepdim=True))
    return d_logits.to(s["logits"].dtype)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    return (xc * rstd[:, None] * s["w"].float() + s["bias"].float()).to(s["x"].dtype), mean, rstd


def _plain_norm_back(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "fp8":
        return _plain_fp8(s)
    if c["op"] == "experts":
        return _plain_experts(s)
    if c["op"] == "route":
        return _plain_route_back(s) if c["back"] else _plain_route(s)
    return _plain_norm_back(s) if c["back"] else _plain_norm(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- exact results
def _exact_codes(x):
    """Codes times scales in 64 bits.  The scale, its inverse and the scaled value are fp32 numbers by
    definition; the code is the nearest of the e4m3 numbers, even at a tie."""
    v = x.view(x.shape[0], -1, 128)
    top = v.double().abs().amax(2, keepdim=True)
    scale = (top / 448.0).float().double()
    inv = torch.where(top > 0, (448.0 / top).float().double(), torch.zeros_like(top))
    u = (v.double() * inv).float().double()
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3.0)
    return ((torch.round(u / step) * step).clamp(-448.0, 448.0) * scale).view(x.shape)


def _exact_weight(q, scale):
    n, d = q.shape
    rows = torch.arange(n, device="cuda") // 128
    return (q.double().view(n, d // 128, 128) * scale.double()[rows][:, :, None]).view(n, d)


def _exact_route_scores(logits, kind):
    if kind == "sigmoid":
        return torch.sigmoid(logits)
    return torch.nan_to_num(torch.softmax(logits, 1), nan=0.0)


def _first_best(v):
    """Best value of each row and the lowest column that has it."""
    best = v.amax(1)
    cols = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return best, torch.where(v == best[:, None], cols, torch.full_like(cols, v.shape[1])).amin(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8":
        x, proj = _exact_codes(s["x"]), s["x"].double() @ s["b"].double().t()
        return [x @ _exact_weight(q, sc).t() + proj @ a.double().t() for q, sc, a in zip(s["q"], s["scale"], s["a"])]
    if op == "experts":
        x, off = _exact_codes(s["x"]), s["offsets"].tolist()
        ys = [torch.empty(s["n_rows"], n, dtype=torch.float64, device="cuda") for n in _rows(case)]
        for e in range(case["n_exp"]):
            j = slice(off[e], off[e + 1])
            t = s["token"][j].long()
            b = s["b"][e] if case["share"] == "expert" else s["b"]
            proj = s["x"][t].double() @ b.double().t()
            for y, q, sc, a in zip(ys, s["q"], s["scale"], s["a"]):
                y[j] = x[t] @ _exact_weight(q[e], sc[e]).t() + proj @ a[e].double().t()
        return ys
    if op == "norm":
        x, w = s["x"].double(), s["w"].double()
        if not case["back"]:
            var, mean = torch.var_mean(x, 1, unbiased=False)
            rstd = torch.rsqrt(var + EPS)
            return (x - mean[:, None]) * rstd[:, None] * w + s["bias"].double(), mean, rstd
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * rstd
        d = case["d"]
        c1, c2 = (dy @ w)[:, None] / d, ((dy * xhat) @ w)[:, None] / d
        return rstd * (dy * w - c1 - xhat * c2), torch.mul(dy, xhat).sum(0), dy.sum(0)
    logits, T, E, k, G = s["logits"].double(), case["T"], case["n_exp"], case["k"], case["groups"]
    score = _exact_route_scores(logits, case["score"])
    rows = torch.arange(T, device="cuda")
    if case["back"]:
        # the Jacobian of each chosen weight, choice by choice
        ids, dw = s["ids"].long(), s["dw"].double()
        pad = torch.cat([score, torch.zeros(T, 1, dtype=torch.float64, device="cuda")], 1)
        col = torch.where(ids < 0, torch.full_like(ids, E), ids)
        p = pad.gather(1, col)
        total = p.sum(1).clamp(min=1e-300) if case["renorm"] else torch.ones(T, dtype=torch.float64, device="cuda")
        d_pad = torch.zeros_like(pad)
        for j in range(k):
            # d w_j = scale (d s_j / total - s_j d total / total^2)
            d_pad[rows, col[:, j]] += SCALE * dw[:, j] / total
            if case["renorm"]:
                for i in range(k):
                    d_pad[rows, col[:, i]] -= SCALE * dw[:, j] * p[:, j] / total ** 2
        d_score = d_pad[:, :E]
        if case["score"] == "sigmoid":
            return d_score * score * torch.sigmoid(-logits)
        return score * d_score - score * (score * d_score).sum(1, keepdim=True)
    sel = score + (0.0 if s["bias"] is None else s["bias"].double())
    sel[logits == -math.inf] = -math.inf
    value = logits.clone() if s["bias"] is None else sel.clone()
    if G > 1:
        by = (value if case["best"] == 1 else sel).view(T, G, E // G)
        stand = by.amax(2)
        if case["best"] == 2 and E // G > 1:
            second = torch.topk(by, 2, dim=2).values[:, :, 1]
            stand = stand + torch.where(second == -math.inf, torch.zeros_like(second), second)
        closed = torch.ones(T, G, dtype=torch.bool, device="cuda")
        for _ in range(case["keep"]):
            at = _first_best(torch.where(closed, stand, torch.full_like(stand, -math.inf)))[1]
            closed[rows, at] = False
        value[closed[:, :, None].expand(T, G, E // G).reshape(T, E)] = -math.inf
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        best, at = _first_best(value)
        some = best > -math.inf
        ids[:, j] = torch.where(some, at, torch.full_like(at, -1)).to(torch.int32)
        w[:, j] = torch.where(some, score[rows, at.clamp(max=E - 1)], torch.zeros_like(best))
        value[rows, at.clamp(max=E - 1)] = -math.inf
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return ids, SCALE * w
