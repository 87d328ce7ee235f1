"""A training step of a mixture-of-experts layer in 32 bits on the library's calls: lists, tokens into expert order,
the caller's expert products, the gated activation, the weighted way back, and every gradient of it through
combine, activation and dispatch.  Against the layer in fp64 with bounds carried from call to call, and against
differences of the fp64 layer."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import glowq, log
from test_gpu_moe_rows import routing

pytestmark = pytest.mark.gpu
U = R.U32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


class Val:
    """A value in fp64 and a bound of the distance of the library's fp32 one from it."""

    def __init__(self, v, e=None):
        self.v, self.e = v, np.zeros_like(v) if e is None else e

    def mm(self, o):
        """Product over L terms in fp32: the factors' errors, and L roundings of sums below sum |a| |b|."""
        a, b = np.abs(self.v), np.abs(o.v)
        e = self.e @ (b + o.e) + a @ o.e
        return Val(self.v @ o.v, e + 1.01 * self.v.shape[1] * U * ((a + self.e) @ (b + o.e)))

    def t(self):
        return Val(self.v.T, self.e.T)

    def __add__(self, o):
        v, e = self.v + o.v, self.e + o.e
        return Val(v, e + U * (np.abs(v) + e))


def silu(g):
    return g / (1.0 + np.exp(-g))


def slope(g):
    s = 1.0 / (1.0 + np.exp(-g))
    return s * (1.0 + g * (1.0 - s))


# |silu'| <= 1.1 and |silu''| <= 1/2 carry an error of the gate; R.GATE is the kernels' own, s (1 + |g| (1 - s)) <= 1.3
def gated(g, u):
    v = silu(g.v) * u.v
    e = 1.1 * g.e * (np.abs(u.v) + u.e) + np.abs(silu(g.v)) * u.e
    return Val(v, e + R.GATE * 1.01 * (np.abs(v) + e) + 1e-36)


def gated_gradients(dh, g, u):
    d, w = np.abs(dh.v) + dh.e, np.abs(u.v) + u.e
    eg = d * w * 0.5 * g.e + 1.1 * (dh.e * w + np.abs(dh.v) * u.e) + R.GATE * 1.3 * 1.01 * d * w + 1e-36
    eu = dh.e * np.abs(silu(g.v)) + d * 1.1 * g.e
    v = dh.v * silu(g.v)
    return Val(dh.v * u.v * slope(g.v), eg), Val(v, eu + R.GATE * 1.01 * (np.abs(v) + eu) + 1e-36)


def layer64(x, w, wg, wu, wd, ids, dy):
    """Loss <dy, y> of the layer from its definition, in fp64 torch on the CPU."""
    y = [x[t] for t in range(x.shape[0])]
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e >= 0:
                g, u = wg[e] @ x[t], wu[e] @ x[t]
                y[t] = y[t] + w[t, j] * (wd[e] @ (g * torch.sigmoid(g) * u))
    return (torch.stack(y) * dy).sum()


@pytest.mark.parametrize("T,k,E,d,f,drop", [(1, 2, 4, 16, 24, 0), (37, 3, 6, 50, 33, 0.3), (130, 2, 8, 64, 48, 0.1)])
def test_training_step(T, k, E, d, f, drop):
    g = glowq()
    gen = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=gen)
    ids = routing(T, k, E, T, drop)
    x, dy, w = rn(T, d), rn(T, d), torch.rand(T, k, generator=gen)
    wg, wu, wd = rn(E, f, d) / d ** 0.5, rn(E, f, d) / d ** 0.5, rn(E, d, f) / f ** 0.5
    log(f"training step T={T} k={k} E={E} d={d} f={f} drop={drop}")
    dev = lambda t: t.cuda()
    xc, dyc, wc, Wg, Wu, Wd = map(dev, (x, dy, w, wg, wu, wd))
    ws = g.init_workspace(torch.empty(g.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda"))

    off, tok, pr = g.moe_sort(dev(ids), E, workspace=ws)
    lo = off.tolist()
    n = T * k  # the lists as they come: rows behind the last expert's have token -1
    part = lambda v, e: v[lo[e]:lo[e + 1]]
    rows = g.moe_dispatch(xc, tok, workspace=ws)
    gate, up, out, dh, drows = (torch.zeros(n, c, device="cuda") for c in (f, f, d, f, d))
    for e in range(E):
        part(gate, e).copy_(part(rows, e) @ Wg[e].t())
        part(up, e).copy_(part(rows, e) @ Wu[e].t())
    h = g.swiglu(gate, up)
    for e in range(E):
        part(out, e).copy_(part(h, e) @ Wd[e].t())
    y = g.moe_combine(out, pr, wc, add=xc, workspace=ws)
    dout, dw = g.moe_combine_backward(dyc, out, pr, tok, wc, workspace=ws)
    for e in range(E):
        part(dh, e).copy_(part(dout, e) @ Wd[e])
    dgate, dup = g.swiglu_backward(dh, gate, up)
    dWg, dWu, dWd = torch.zeros_like(Wg), torch.zeros_like(Wu), torch.zeros_like(Wd)
    for e in range(E):
        part(drows, e).copy_(part(dgate, e) @ Wg[e] + part(dup, e) @ Wu[e])
        dWg[e], dWu[e] = part(dgate, e).t() @ part(rows, e), part(dup, e).t() @ part(rows, e)
        dWd[e] = part(dout, e).t() @ part(h, e)
    dx = g.moe_dispatch_backward(drows, pr, workspace=ws) + dyc
    assert g.workspace_status(ws) == g.OK
    live = lo[E]
    for v in (rows, h, dout, dgate, dup):
        assert not v[live:].any()

    # the same calls in fp64, each with the bound of what came before it
    ro, rt, rp = R.sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(tok.cpu().numpy(), rt)
    assert np.array_equal(pr.cpu().numpy(), rp)
    x64, dy64, w64 = R.f64(x), R.f64(dy), R.f64(w)
    G, D = {}, {k_: np.zeros((n, c)) for k_, c in (("o", d), ("eo", d), ("r", d), ("er", d))}
    dwv, dwe = np.zeros((T, k)), np.zeros((T, k))
    pairs = {int(rp[t, j]): (t, j) for t in range(T) for j in range(k) if rp[t, j] >= 0}
    for e in range(E):
        a, b = lo[e], lo[e + 1]
        if a == b:
            continue
        at = [pairs[i] for i in range(a, b)]
        X = Val(np.stack([x64[t] for t, _ in at]))
        A, B, C = Val(R.f64(wg[e])), Val(R.f64(wu[e])), Val(R.f64(wd[e]))
        ge, ue = X.mm(A.t()), X.mm(B.t())
        he = gated(ge, ue)
        oe = he.mm(C.t())
        D["o"][a:b], D["eo"][a:b] = oe.v, oe.e
        do = np.stack([w64[t, j] * dy64[t] for t, j in at])
        do = Val(do, U * np.abs(do))
        for i, (t, j) in enumerate(at):
            dwv[t, j] = dy64[t] @ oe.v[i]
            dwe[t, j] = np.abs(dy64[t]) @ (oe.e[i] + 1.01 * (d + 1) * U * (np.abs(oe.v[i]) + oe.e[i]))
        dhe = do.mm(C)
        dge, due = gated_gradients(dhe, ge, ue)
        dr = dge.mm(A) + due.mm(B)
        D["r"][a:b], D["er"][a:b] = dr.v, dr.e
        G[e] = (dge.t().mm(X), due.t().mm(X), do.t().mm(he))
    ref = {"y": (x64.copy(), np.zeros_like(x64)), "dx": (dy64.copy(), np.zeros_like(x64))}
    mag = {"y": np.abs(x64), "dx": np.abs(dy64)}
    for row, (t, j) in pairs.items():
        for name, c, v, e in (("y", w64[t, j], D["o"][row], D["eo"][row]), ("dx", 1.0, D["r"][row], D["er"][row])):
            ref[name][0][t] += c * v
            ref[name][1][t] += c * e
            mag[name][t] += c * (np.abs(v) + e)
    for name, got in (("y", y), ("dx", dx)):
        R.within(got, ref[name][0], ref[name][1] + 1.01 * (k + 2) * U * mag[name] + 1e-36, name)
    R.within(dw, dwv, dwe + 1e-36, "dw")
    for e in range(E):
        for name, got, i in (("dWg", dWg, 0), ("dWu", dWu, 1), ("dWd", dWd, 2)):
            if e in G:
                R.within(got[e], G[e][i].v, G[e][i].e + 1e-36, f"{name}[{e}]")
            else:
                assert not got[e].any()

    # differences of the definition: central, at step s along random directions; third-order terms fall as s^2, so
    # two steps a factor of two apart leave the extrapolated value (4 D(s/2) - D(s)) / 3 off by order s^4
    names = ("x", "w", "wg", "wu", "wd")
    base = [t.double() for t in (x, w, wg, wu, wd)]
    grads = [t.cpu().double() for t in (dx, dw, dWg, dWu, dWd)]
    for i, name in enumerate(names):
        v = rn(*base[i].shape).double()
        v /= v.norm()

        def diff(s):
            f_ = lambda c: float(layer64(*[b + c * v if q == i else b for q, b in enumerate(base)], ids, dy.double()))
            return (f_(s) - f_(-s)) / (2 * s)
        d1, d2 = diff(1e-2), diff(5e-3)
        num = (4 * d2 - d1) / 3
        got = float((grads[i] * v).sum())
        # the fp32 gradients within 2^-12 of the sum of their products' sizes (their bounds above are far below), the
        # differences within a tenth of what the extrapolation moved, and fp64 rounding over the step
        tol = 2.0 ** -12 * float((grads[i] * v).abs().sum()) + 0.1 * abs(d2 - d1) + 1e-9 * float(dy.abs().sum())
        print(f"  {name}: {got:.6f} against {num:.6f}, allowed {tol:.2e}", flush=True)
        assert abs(got - num) <= tol, name
