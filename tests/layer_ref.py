"""Plain fp64 references (numpy) of the 8-bit integer group product, the routed rows and the gated
activation, with elementwise error bounds: every bound counts the roundings the library documents
(fp32 sums, one rounding to the output type), from eps / 2 of each type."""
import numpy as np
import torch

from oracle import glowq_ref as G

U32 = 2.0 ** -24              # half a step of fp32, relative
HALF = {"f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half a step of the subnormals


def f64(t):
    return t.detach().cpu().double().numpy()


def w8a8(x, codes, scales, b, a_list, correct):
    """(outputs, bounds): s_t s[o] sum_k c[t, k] q[o, k] + R A^T with exact integer sums.  Bound: the
    sum's conversion and two scalings in fp32, R's fp32 sum over d and its rounding to fp16, the
    fp32 sum over r, the final rounding."""
    c, s = G.quantize_x_int8(x)
    xf = f64(x)
    outs, bounds = [], []
    for i, (q, sc) in enumerate(zip(codes, scales)):
        y = (c.astype(np.float64) @ f64(q).T) * s.astype(np.float64)[:, None] * f64(sc)[None, :]
        err = 3 * U32 * np.abs(y)
        if correct:
            bf, af = f64(b), f64(a_list[i])
            R = xf @ bf.T
            d, r = xf.shape[1], bf.shape[0]
            absR = np.abs(xf) @ np.abs(bf).T
            dR = d * U32 * absR * 1.01 + HALF["f16"] * np.abs(R) + TINY["f16"]
            corr = R @ af.T
            y = y + corr
            err = err + dR @ np.abs(af).T * 1.01 + (r + 1) * U32 * (np.abs(R) @ np.abs(af).T + np.abs(y)) * 1.01
        outs.append(y)
        bounds.append(err * 1.01 + HALF["f16"] * (np.abs(y) + err) + TINY["f16"])
    return outs, bounds


def sort(ids, n_exp):
    """Lists of ids [T][k] by the definition: pairs in order, expert after expert."""
    T, k = ids.shape
    flat = [int(v) for v in ids.reshape(-1)]
    token, pair_row = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
    offsets = [0]
    by = {e: [] for e in range(n_exp)}
    for p, e in enumerate(flat):
        if 0 <= e < n_exp:
            by[e].append(p)
    row = 0
    for e in range(n_exp):
        for p in by[e]:
            token[row], pair_row[p] = p // k, row
            row += 1
        offsets.append(row)
    return np.array(offsets, np.int32), token, pair_row.reshape(T, k)


def combine(rows, pair_row, w, add, kind):
    rf = f64(rows)
    T, k = pair_row.shape
    y = np.zeros((T, rf.shape[1])) if add is None else f64(add).copy()
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            p = int(pair_row[t, j])
            if p >= 0:
                v = (1.0 if w is None else float(w[t, j])) * rf[p]
                y[t] += v
                mag[t] += np.abs(v)
    err = (k + 1) * U32 * mag * 1.01
    return y, err + HALF[kind] * (np.abs(y) + err) + TINY[kind]


def combine_backward(dy, rows, pair_row, w, n_rows, kind):
    """(d_rows, bound, dw, bound, named rows)."""
    g, rf = f64(dy), f64(rows)
    T, k = pair_row.shape
    d = g.shape[1]
    dr, dw, dwb = np.zeros((n_rows, d)), np.zeros((T, k)), np.zeros((T, k))
    named = np.zeros(n_rows, bool)
    for t in range(T):
        for j in range(k):
            p = int(pair_row[t, j])
            if p >= 0:
                dr[p] = (1.0 if w is None else float(w[t, j])) * g[t]
                named[p] = True
                dw[t, j] = float(g[t] @ rf[p])
                dwb[t, j] = (d + 1) * U32 * float(np.abs(g[t]) @ np.abs(rf[p])) * 1.01
    drb = U32 * np.abs(dr)
    return dr, drb + HALF[kind] * (np.abs(dr) + drb) + TINY[kind], dw, dwb + 2.0 ** -150, named


# exp within two steps of fp32, one quotient, up to three products: under 2^-20 relative in all
GATE = 2.0 ** -20
FLUSH = 2.0 ** -126  # sigmoids below the smallest normal number may lose all their bits


def swiglu(gate, up, kind):
    g, u = f64(gate), f64(up)
    with np.errstate(over="ignore", invalid="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        h = g * s * u
    err = GATE * np.abs(h) + np.abs(g * u) * FLUSH
    return h, err + HALF[kind] * (np.abs(h) + err) + TINY[kind]


def swiglu_backward(dh, gate, up, kind):
    d, g, u = f64(dh), f64(gate), f64(up)
    with np.errstate(over="ignore", invalid="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        t = 1.0 / (1.0 + np.exp(g))
    dg, du = d * u * s * (1.0 + g * t), d * g * s
    # 1 + g t cancels near g = -1.28: its error is that of its terms
    eg = GATE * np.abs(d * u * s) * (1.0 + np.abs(g * t)) + np.abs(d * u) * (1.0 + np.abs(g)) * FLUSH
    eu = GATE * np.abs(du) + np.abs(d * g) * FLUSH
    half, tiny = HALF[kind], TINY[kind]
    return (dg, eg + half * (np.abs(dg) + eg) + tiny), (du, eu + half * (np.abs(du) + eu) + tiny)


def within(got, ref, bound, what):
    """Every value within its bound; fp16 results from 65520 on (the largest number, 65504, plus half
    its step of 32) are infinities by rounding."""
    if got.dtype == torch.float16:
        ref = np.where(np.abs(ref) >= 65520.0, np.copysign(np.inf, ref), ref)
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    far = np.isinf(ref)
    assert np.array_equal(got[far], ref[far]), what
    got, ref, bound = got[~far], ref[~far], bound[~far]
    bad = ~(np.abs(got - ref) <= bound)
    worst = float(np.max(np.abs(got - ref) / bound)) if got.size else 0.0
    print(f"  {what}: largest error {worst:.3f} of the bound", flush=True)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), worst)
