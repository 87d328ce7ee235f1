"""The 8-bit integer group product and the operators around the mixture-of-experts product, as
measured workloads: their cases, inputs, plain forms, calls and exact results.

w8a8       y_i = s_t s_i[o] sum_k c[t, k] q_i[o, k] + (X B^T) A_i^T, with per-token codes
           c = clamp(round_half_even(x / s_t), -127, 127), s_t = max |x_t| / 127 (fp32)
sort       expert ids [T][k] -> rows listed by expert (offsets, token of each row, row of each
           (token, choice) pair), pairs of one expert in their order; id -1 takes no row
dispatch   rows[j] = x[row_token[j]] and its gradient dx[t] = sum_j d_rows[pair_row[t, j]]
combine    y[t] = add[t] + sum_j w[t, j] rows[pair_row[t, j]] and its gradients
           d_rows[pair_row[t, j]] = w[t, j] dy[t], dw[t, j] = <dy[t], rows[pair_row[t, j]]>
swiglu     h = g sigmoid(g) u and its gradients

With `own` false run() computes the plain forms in elementary torch operations; with `own` true it
calls the library.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def _w8a8(T, d, rows, r, name=None):
    c = {"op": "w8a8", "T": T, "d": d, "rows": ",".join(str(n) for n in rows), "r": r}
    return {"name": name, **c} if name else c


def _moe(op, back, T, k, n_exp, d, dtype, drop, add, name=None):
    c = {"op": op, "back": back, "T": T, "k": k, "n_exp": n_exp, "d": d, "dtype": dtype, "drop": drop, "add": add}
    return {"name": name, **c} if name else c


def _swiglu(back, rows, f, dtype, name=None):
    c = {"op": "swiglu", "back": back, "rows": rows, "d": f, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one generated token through the Q/K/V group of an 8B decoder (grouped-query heads)
        _w8a8(1, 4096, (4096, 1024, 1024), 64, "w8a8_qkv_t1"),
        # a small ragged batch through one expert's gate/up pair
        _w8a8(37, 2048, (1408, 1408), 64, "w8a8_gateup_t37"),
        # a short prompt through the long-row down projection
        _w8a8(512, 14336, (4096,), 64, "w8a8_down_t512"),
        # a 2048-token prompt through gate/up
        _w8a8(2048, 4096, (11008, 11008), 64, "w8a8_gateup_t2048"),
        # routing lists of one generated token (latency)
        _moe("sort", False, 1, 4, 60, 0, "f16", 0, False, "sort_t1"),
        # routing lists of a large prompt batch, one pair in 16 without an expert
        _moe("sort", False, 65536, 4, 60, 0, "f16", 16, False, "sort_t65536"),
        # token rows into expert order at an odd prompt length
        _moe("dispatch", False, 2047, 4, 60, 2048, "f16", 0, False, "dispatch_t2047"),
        # the gradient of that at a training batch, in 32 bits
        _moe("dispatch", True, 4096, 4, 60, 2048, "f32", 0, False, "dispatch_back_t4096_f32"),
        # expert outputs back to tokens, weighted, onto the shared expert's output
        _moe("combine", False, 16384, 4, 60, 2048, "f16", 0, True, "combine_t16384"),
        # its gradients at an odd batch, one pair in 16 without an expert
        _moe("combine", True, 8191, 4, 60, 2048, "f16", 16, False, "combine_back_t8191"),
        # the gated activation of one token's four routed rows (latency)
        _swiglu(False, 4, 1408, "f16", "swiglu_rows4"),
        # its gradients at a training batch, in 32 bits
        _swiglu(True, 16383, 1408, "f32", "swiglu_back_rows16383_f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w8a8", "w8a8", "sort", "dispatch", "combine", "combine", "swiglu"])
    if op == "w8a8":
        while True:
            T, d = _spread(rng, 1, 4096), 128 * _spread(rng, 1, 112)
            rows = tuple(_spread(rng, 1, 16384) for _ in range(rng.randint(1, 3)))
            if T * d * sum(rows) <= 2048 * 4096 * 22016:
                return _w8a8(T, d, rows, rng.choice([0, 8, 24, 64, 128, 256]))
    back = op != "sort" and rng.random() < 0.5
    dtype = rng.choice(["f16", "f16", "f32"])
    if op == "swiglu":
        return _swiglu(back, _spread(rng, 1, 16383), _spread(rng, 16, 1408), dtype)
    n_exp = _spread(rng, 2, 256)
    k = rng.randint(1, min(8, n_exp))
    drop = rng.choice([0, 0, 4, 16])
    if op == "sort":
        return _moe(op, False, _spread(rng, 1, 262144 // k), k, n_exp, 0, "f16", drop, False)
    while True:
        T, d = _spread(rng, 1, 16384), _spread(rng, 16, 4096)
        if T * k * d * (2 if dtype == "f32" else 1) <= (16384 if op == "combine" else 8192) * 4 * 2048:
            return _moe(op, back, T, k, n_exp, d, dtype, drop, op == "combine" and not back and rng.random() < 0.5)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] == "w8a8":
        T, d, r, n = case["T"], case["d"], case["r"], sum(_rows(case))
        return {"bytes": 2 * T * d + n * d + 4 * n + 2 * r * (d + n) + 2 * T * n,
                "flops": 2 * T * n * d + 2 * r * T * (d + n)}
    e = 2 if case["dtype"] == "f16" else 4
    if case["op"] == "swiglu":
        n = case["rows"] * case["d"]
        return {"bytes": (5 if case["back"] else 3) * n * e, "flops": (12 if case["back"] else 5) * n}
    n = case["T"] * case["k"]
    if case["op"] == "sort":
        return {"bytes": 12 * n + 4 * (case["n_exp"] + 1), "flops": n}
    live = n - (n // case["drop"] if case["drop"] else 0)
    tokens, pairs = case["T"] * case["d"], live * case["d"]
    if case["op"] == "dispatch":
        return {"bytes": (tokens + pairs) * e + 4 * n, "flops": pairs if case["back"] else 0}
    if case["back"]:
        return {"bytes": (tokens + 2 * pairs) * e + 12 * n + 4 * live, "flops": 3 * pairs}
    return {"bytes": (tokens * (2 if case["add"] else 1) + pairs) * e + 8 * n, "flops": 2 * pairs}


# --------------------------------------------------------------------------- inputs
def _rows(case):
    return [int(n) for n in case["rows"].split(",")]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "w8a8":
        T, d, r = case["T"], case["d"], case["r"]
        # activations with a power-law channel spectrum; weights with a few outlier input columns
        chan = torch.arange(1, d + 1, device="cuda").float() ** -0.5
        chan = (chan * math.sqrt(d) / chan.norm())[torch.randperm(d, generator=gen, device="cuda")]
        s["x"] = (_randn(gen, T, d) * chan).half()
        s["q"], s["scale"], s["a"] = [], [], []
        for n in _rows(case):
            w = 0.02 * _randn(gen, n, d)
            w[:, : min(4, d)] *= 10.0
            sc = w.abs().amax(1) / 127.0
            s["q"].append(torch.round(w / sc[:, None]).clamp(-127, 127).to(torch.int8))
            s["scale"].append(sc)
            s["a"].append((_randn(gen, n, r) * (0.02 * 0.03 * math.sqrt(d / max(r, 1)))).half())
        s["b"] = (_randn(gen, r, d) / math.sqrt(d)).half()
    elif case["op"] == "swiglu":
        n, f, t = case["rows"], case["d"], DTYPES[case["dtype"]]
        s["gate"], s["up"] = (2.0 * _randn(gen, n, f)).to(t), _randn(gen, n, f).to(t)
        if case["back"]:
            s["dh"] = _randn(gen, n, f).to(t)
    else:
        T, k, E, d, t = case["T"], case["k"], case["n_exp"], case["d"], DTYPES[case["dtype"]]
        # distinct experts per token from scores with a per-expert bias (some experts are busier)
        score = _randn(gen, T, E) + 0.7 * _randn(gen, 1, E)
        top = torch.topk(score, k, dim=1)
        ids = top.indices.to(torch.int32)
        if case["drop"]:
            gone = torch.randperm(T * k, generator=gen, device="cuda")[: T * k // case["drop"]]
            ids.view(-1)[gone] = -1
        s["ids"], s["n_exp"] = ids, E
        if case["op"] != "sort":
            offsets, token, pair_row = _plain_sort(ids, E)
            n_rows = int(offsets[-1])
            s["token"], s["pair_row"], s["n_rows"] = token[:n_rows].contiguous(), pair_row, n_rows
            s["w"] = torch.softmax(top.values, 1)
            if case["op"] == "dispatch":
                s["rows" if case["back"] else "x"] = _randn(gen, n_rows if case["back"] else T, d).to(t)
            else:
                s["rows"] = _randn(gen, n_rows, d).to(t)
                if case["back"]:
                    s["dy"] = _randn(gen, T, d).to(t)
                elif case["add"]:
                    s["add"] = _randn(gen, T, d).to(t)
    if own:
        s["plan"] = _plan(s)
    return s


# --------------------------------------------------------------------------- the library's calls
def _plan(s):
    """What a program keeps between calls: weights in the device layout, a workspace."""
    from rank_error_compensation_amd import glowq as g
    c = s["case"]
    if c["op"] == "w8a8":
        w = [g.QWeight.from_int8(q, sc) for q, sc in zip(s["q"], s["scale"])]
        n = g.w8a8_workspace_bytes(c["T"], c["d"], c["r"])
        return g, w, torch.empty(n, dtype=torch.uint8, device="cuda")
    if c["op"] == "swiglu":
        return g, None, None
    n = g.moe_sort_workspace_bytes(c["T"], c["k"], c["n_exp"])
    return g, None, g.init_workspace(torch.empty(n, dtype=torch.uint8, device="cuda"))


def _run_own(s):
    c = s["case"]
    g, weights, ws = s["plan"]
    if c["op"] == "w8a8":
        return g.group_forward_w8a8(s["x"], weights, s["b"] if c["r"] else None, s["a"] if c["r"] else [], c["r"],
                                    c["r"] > 0, workspace=ws)
    if c["op"] == "sort":
        return g.moe_sort(s["ids"], s["n_exp"], workspace=ws)
    if c["op"] == "dispatch":
        if c["back"]:
            return g.moe_dispatch_backward(s["rows"], s["pair_row"], workspace=ws)
        return g.moe_dispatch(s["x"], s["token"], workspace=ws)
    if c["op"] == "combine":
        if c["back"]:
            return g.moe_combine_backward(s["dy"], s["rows"], s["pair_row"], s["token"], s["w"], workspace=ws)
        return g.moe_combine(s["rows"], s["pair_row"], s["w"], add=s.get("add"), workspace=ws)
    if c["back"]:
        return g.swiglu_backward(s["dh"], s["gate"], s["up"])
    return g.swiglu(s["gate"], s["up"])


# --------------------------------------------------------------------------- plain forms
def _plain_sort(ids, n_exp):
    T, k = ids.shape
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, n_exp), flat)
    key, order = torch.sort(key, stable=True)
    n = T * k
    row = torch.arange(n, device=ids.device, dtype=torch.int32)
    live = key < n_exp
    token = torch.where(live, (order // k).to(torch.int32), torch.full_like(row, -1))
    pair_row = torch.empty_like(row)
    pair_row[order] = torch.where(live, row, torch.full_like(row, -1))
    offsets = torch.searchsorted(key, torch.arange(n_exp + 1, device=ids.device, dtype=torch.int32)).to(torch.int32)
    return offsets, token, pair_row.reshape(T, k)


def _gathered(rows, pair_row):
    """fp32 [T][k][d] rows of every pair, zero where a pair has none."""
    v = rows[pair_row.clamp(min=0).long()].float()
    return torch.where((pair_row >= 0)[..., None], v, torch.zeros_like(v))


def _plain_w8a8(s):
    x = s["x"].float()
    scale = x.abs().amax(1, keepdim=True)
    scale = scale / torch.full_like(scale, 127.0)
    codes = torch.where(scale > 0, torch.round(x / scale).clamp(-127.0, 127.0), torch.zeros_like(x))
    proj = x @ s["b"].float().t()
    return [((codes @ q.float().t()) * scale * sc + proj @ a.float().t()).half()
            for q, sc, a in zip(s["q"], s["scale"], s["a"])]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "w8a8":
        return _plain_w8a8(s)
    if c["op"] == "sort":
        return _plain_sort(s["ids"], s["n_exp"])
    if c["op"] == "dispatch":
        if c["back"]:
            return _gathered(s["rows"], s["pair_row"]).sum(1).to(s["rows"].dtype)
        return s["x"][s["token"].long()]
    if c["op"] == "combine":
        v = _gathered(s["rows"], s["pair_row"])
        if c["back"]:
            dy = s["dy"].float()[:, None]
            d_rows = torch.empty(s["n_rows"] + 1, v.shape[2], dtype=s["rows"].dtype, device=v.device)
            slot = torch.where(s["pair_row"] < 0, torch.full_like(s["pair_row"], s["n_rows"]), s["pair_row"])
            d_rows[slot.long()] = (s["w"][..., None] * dy).to(d_rows.dtype)
            return d_rows[: s["n_rows"]], (v * dy).sum(2)
        y = (s["w"][..., None] * v).sum(1)
        return (y + s["add"].float() if "add" in s else y).to(s["rows"].dtype)
    g, u = s["gate"].float(), s["up"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    if c["back"]:
        dh = s["dh"].float()
        return (dh * u * sg * (1.0 + g * (1.0 - sg))).to(s["gate"].dtype), (dh * g * sg).to(s["gate"].dtype)
    return (g * sg * u).to(s["gate"].dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- exact results
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        # rank of a pair within its expert: earlier pairs that name the same expert
        ids = s["ids"].cpu().reshape(-1)
        n, E, k = ids.numel(), case["n_exp"], case["k"]
        counts = torch.tensor([int((ids == e).sum()) for e in range(E)])
        start = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
        token = torch.full((n,), -1, dtype=torch.int32)
        pair_row = torch.full((n,), -1, dtype=torch.int32)
        for e in range(E):
            p = (ids == e).nonzero().reshape(-1)
            token[start[e]:start[e + 1]] = (p // k).to(torch.int32)
            pair_row[p] = torch.arange(int(start[e]), int(start[e + 1]), dtype=torch.int32)
        return start.to(torch.int32), token, pair_row.reshape(-1, k)
    if op == "w8a8":
        x = s["x"].double()
        # the scale and the quotient are fp32 values by definition; their 64-bit forms round to them
        scale = (x.abs().amax(1, keepdim=True) / 127.0).float().double()
        codes = torch.round((x / scale).float()).double().nan_to_num(0.0).clamp(-127, 127)
        proj = x @ s["b"].double().t()
        return [scale * (codes @ q.double().t()) * sc.double() + proj @ a.double().t()
                for q, sc, a in zip(s["q"], s["scale"], s["a"])]
    if op == "swiglu":
        g, u = s["gate"].double(), s["up"].double()
        sg = torch.reciprocal(1.0 + torch.exp(-g))
        if case["back"]:
            dh = s["dh"].double()
            return dh * u * (sg + g * sg * (1.0 - sg)), dh * (g * sg)
        return g * sg * u
    if op == "dispatch" and not case["back"]:
        return s["x"].double().index_select(0, s["token"].long())
    # tokens take their rows one choice at a time
    T, k, d = case["T"], case["k"], case["d"]
    pair_row, rows = s["pair_row"].long(), s["rows"].double()
    rows = torch.cat([rows, torch.zeros(1, d, dtype=torch.float64, device="cuda")])  # row -1: nothing
    if op == "combine" and case["back"]:
        dy, w = s["dy"].double(), s["w"].double()
        d_rows = torch.zeros_like(rows)
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            d_rows[pair_row[:, j]] = w[:, j, None] * dy
            dw[:, j] = (rows[pair_row[:, j]] * dy).sum(1)
        return d_rows[:-1], dw
    y = s["add"].double() if "add" in s else torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        v = rows[pair_row[:, j]]
        y = y + (s["w"][:, j, None].double() * v if op == "combine" else v)
    return y
