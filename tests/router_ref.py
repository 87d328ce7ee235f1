"""Plain fp64 references (numpy) of the router and the layer norm, with elementwise error bounds that count the
roundings the library documents (fp32 sums, one rounding to the output type), from eps / 2 of each type."""
import math

import numpy as np

from layer_ref import HALF, TINY, U32, f64


# --------------------------------------------------------------------------- router
def scores(row, score):
    """fp64 scores of one token; experts of logit -inf have 0."""
    live = row > -np.inf
    s = np.zeros(row.size)
    if score == "sigmoid":
        e = np.exp(-np.abs(row[live]))
        s[live] = np.where(row[live] >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    elif live.any():
        e = np.exp(row[live] - row[live].max())
        s[live] = e / e.sum()
    return s


def choose(row, k, score, bias, n_group, keep, best):
    """Expert ids of one token by the definition."""
    E = row.size
    s = scores(row, score) + (0.0 if bias is None else bias)
    s = np.where(row == -np.inf, -np.inf, s)
    value = row.copy() if bias is None else s.copy()
    if keep < n_group:
        n = E // n_group
        stand = []
        for g in range(n_group):
            by = sorted((value if best == 1 else s)[g * n:(g + 1) * n], reverse=True)
            top = [v for v in by[:best] if v > -np.inf]
            stand.append(sum(top) if top else -np.inf)
        order = sorted(range(n_group), key=lambda g: (-stand[g], g))
        for g in order[keep:]:
            value[g * n:(g + 1) * n] = -np.inf
    ids = []
    for _ in range(k):
        e = int(np.argmax(value))  # the first of equal values
        if value[e] == -np.inf:
            ids.append(-1)
        else:
            ids.append(e)
            value[e] = -np.inf
    return ids


def spread(row):
    """Counts of fp32 steps in a softmax of this row: exp's argument rounds by |l - top| steps, the sum by one
    a term in a chain (at most 20), exp and the quotient by a few."""
    live = row[np.isfinite(row)]
    return 64.0 + 4.0 * (float(live.max() - live.min()) if live.size else 0.0)


def route(logits, k, score, bias, n_group, keep, best, renorm, scale):
    """(ids, weights, bounds)."""
    lo = f64(logits)
    b = None if bias is None else f64(bias)
    T = lo.shape[0]
    ids, w, bound = np.full((T, k), -1, np.int32), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        if np.isnan(lo[t]).any() or (lo[t] == np.inf).any() or (b is not None and (np.isnan(b).any() or (b == np.inf).any())):
            continue
        ids[t] = choose(lo[t], k, score, b, n_group, keep, best)
        w[t] = weights(lo[t], ids[t], score, renorm, scale)
        bound[t] = U32 * spread(lo[t]) * np.abs(w[t]) + abs(scale) * 2.0 ** -126
    return ids, w, bound


def weights(row, ids, score, renorm, scale):
    live = ids >= 0
    out = np.zeros(ids.size)
    if not live.any():
        return out
    l = row[ids[live]]
    if renorm:
        if score == "sigmoid":  # log sigmoid: ratios of scores too small for a number
            l = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
        e = np.exp(l - l.max())
        out[live] = scale * e / e.sum()
    else:
        out[live] = scale * scores(row, score)[ids[live]]
    return out


def route_backward(dw, logits, ids, score, renorm, scale, kind):
    """(d_logits, bound)."""
    lo, g, chosen = f64(logits), f64(dw), ids.cpu().numpy()
    T, E = lo.shape
    k = chosen.shape[1]
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = scores(lo[t], score)
        live = [j for j in range(k) if 0 <= chosen[t, j] < E and lo[t, chosen[t, j]] > -np.inf]
        e = [int(chosen[t, j]) for j in live]
        d = np.array([g[t, j] for j in live])
        steps = U32 * (spread(lo[t]) + k)
        mag = np.zeros(E)
        if renorm:
            l = lo[t, e] if score == "softmax" else np.minimum(lo[t, e], 0) - np.log1p(np.exp(-np.abs(lo[t, e])))
            a = np.exp(l - l.max()) / np.exp(l - l.max()).sum() if e else np.zeros(0)
            c, cm = float(a @ d), float(a @ np.abs(d))
            for j, x in enumerate(e):
                slope = 1.0 if score == "softmax" else float(scores(-lo[t, x:x + 1], "sigmoid")[0])
                out[t, x] += scale * a[j] * (d[j] - c) * slope
                mag[x] += abs(scale) * a[j] * (abs(d[j]) + cm) * slope
        elif score == "softmax":
            sums, sm = np.zeros(E), np.zeros(E)
            for j, x in enumerate(e):
                sums[x] += d[j]
                sm[x] += abs(d[j])
            dot, dm = float(s[e] @ d), float(s[e] @ np.abs(d))
            out[t] = scale * s * (sums - dot)
            mag = abs(scale) * s * (sm + dm)
        else:
            for j, x in enumerate(e):
                slope = s[x] * float(scores(-lo[t, x:x + 1], "sigmoid")[0])
                out[t, x] += scale * d[j] * slope
                mag[x] += abs(scale * d[j]) * slope
        bound[t] = steps * mag + 2.0 ** -126 * abs(scale) * (1 + np.abs(g[t]).sum())
    return out, bound + HALF[kind] * (np.abs(out) + bound) + TINY[kind]


# --------------------------------------------------------------------------- layer norm
CHAIN = 32 + 16  # additions one value passes in a row's fp32 sum: 32 in a thread, then pairs and wavefronts


def norm(x, w, b, eps, kind):
    """((y, bound), (mean, bound), (rstd, bound))."""
    xf = f64(x)
    T, d = xf.shape
    wf = np.ones(d) if w is None else f64(w)
    bf = np.zeros(d) if b is None else f64(b)
    eps = float(np.float32(eps))
    mean = xf.mean(1)
    e_mean = (CHAIN + 1) * U32 * np.abs(xf).mean(1)
    c = xf - mean[:, None]
    var = (c * c).mean(1)
    # around a mean that is off by e: the variance grows by e^2, each square by 2 e |c| and three steps
    e_var = (CHAIN + 4) * U32 * var + 2 * e_mean ** 2 + U32 * (var + eps)
    rstd = 1.0 / np.sqrt(var + eps)
    r_rel = e_var / (var + eps) / 2 * 1.1 + 3 * U32
    xh = c * rstd[:, None]
    y = xh * wf + bf
    err = np.abs(wf) * rstd[:, None] * (e_mean[:, None] + U32 * np.abs(c)) * 1.1
    err = err + np.abs(xh * wf) * (r_rel[:, None] + 3 * U32) * 1.1 + U32 * (np.abs(y) + np.abs(bf))
    return ((y, err + HALF[kind] * (np.abs(y) + err) + TINY[kind]), (mean, e_mean + 2.0 ** -149),
            (rstd, rstd * r_rel * 1.01))


def norm_backward(dy, x, mean, rstd, w, kind):
    """((dx, bound), (dw, bound), (db, bound)) for the given fp32 mean and rstd."""
    g0, xf, mu, rs = f64(dy), f64(x), f64(mean)[:, None], f64(rstd)[:, None]
    T, d = xf.shape
    wf = np.ones(d) if w is None else f64(w)
    xh, g = (xf - mu) * rs, g0 * wf
    c1, c2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    dx = rs * (g - c1 - xh * c2)
    e1 = (CHAIN + 3) * U32 * np.abs(g).mean(1, keepdims=True)
    e2 = (CHAIN + 6) * U32 * np.abs(g * xh).mean(1, keepdims=True)
    err = rs * (5 * U32 * np.abs(g) + e1 + 3 * U32 * np.abs(c1) + np.abs(xh) * (e2 + 6 * U32 * np.abs(c2))) * 1.01 + U32 * np.abs(dx)
    # additions: rows in turn in a team (a 256th of them at most), a workgroup's teams (1024 threads in 16s: 64 at most), then up
    # to 16 workgroups' sums in a wavefront and 16 wavefronts; 6 steps of the term itself
    chain = -(-T // 256) + 64 + 16 + 16 + 6
    dw, db = (g0 * xh).sum(0), g0.sum(0)
    return ((dx, err + HALF[kind] * (np.abs(dx) + err) + TINY[kind]),
            (dw, chain * U32 * np.abs(g0 * xh).sum(0) + 2.0 ** -149), (db, chain * U32 * np.abs(g0).sum(0) + 2.0 ** -149))
