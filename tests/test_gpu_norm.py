"""Layer norm and its gradients against plain fp64 references and differences."""
import numpy as np
import pytest
import torch

import layer_ref as R
import router_ref as Q
from gpu_util import glowq, log

pytestmark = pytest.mark.gpu
KINDS = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


def made(T, d, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    x = rn(T, d) * (0.3 + rn(1, d).abs()) + 2.0 * rn(T, 1)
    return [t.to(KINDS[kind]).cuda() for t in (x, 1 + 0.3 * rn(d), 0.2 * rn(d), rn(T, d))]


# every form (columns up to 128, 256, 512, ... 16384), one column, rows that are no multiple of 16 bytes, one row to
# more rows than workgroups of every form take at once
SHAPES = [(1, 1), (3, 2), (5, 7), (1, 8), (70, 64), (33, 100), (17, 128), (40, 129), (9, 250), (33, 256), (6, 257), (11, 500),
          (515, 512), (7, 1000), (3, 1024), (300, 1025), (33, 2047), (515, 2048), (2, 2050), (1, 4096), (600, 4095), (3, 5001),
          (19, 8192), (2, 11008), (5, 16383), (270, 16384), (9000, 16), (4500, 130), (0, 128)]


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_and_gradients(shape, kind):
    g = glowq()
    T, d = shape
    log(f"norm {shape} {kind}")
    x, w, b, dy = made(T, d, kind, T + d)
    for ww, bb in ((w, b), (None, None), (w, None), (None, b)):
        y, mean, rstd = g.layer_norm(x, ww, bb, 1e-5)
        (ry, by), (rm, bm), (rr, br) = Q.norm(x, ww, bb, 1e-5, kind)
        R.within(y, ry, by, "y")
        R.within(mean, rm, bm, "mean")
        R.within(rstd, rr, br, "rstd")
        if bb is not None:
            continue
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, ww)
        (rx, bx), (rw, bw), (rb, bb_) = Q.norm_backward(dy, x, mean, rstd, ww, kind)
        R.within(dx, rx, bx, "dx")
        R.within(dw, rw, bw, "dw")
        R.within(db, rb, bb_, "db")


def test_rows_of_one_value_far_means_and_odd_values():
    """No variance (rstd = 1 / sqrt(eps)), a mean 1000 times the deviation, infinities and NaN in one row only."""
    g = glowq()
    for kind in ("f16", "f32"):
        x, w, b, dy = made(6, 300, kind, 1)
        x[0] = 3.0
        x[1] = 0.0
        x[2] = x[2] * 0.01 + 30.0
        y, mean, rstd = g.layer_norm(x, w, b, 1e-5)
        for got, (ref, bound), name in zip((y, mean, rstd), Q.norm(x, w, b, 1e-5, kind), ("y", "mean", "rstd")):
            R.within(got, ref, bound, name)
        x[4, 7], x[5, 0] = float("inf"), float("nan")
        y2, m2, r2 = g.layer_norm(x, w, b, 1e-5)
        assert torch.equal(y2[:4], y[:4]) and torch.isnan(y2[4:]).all()
        dx, dw, db = g.layer_norm_backward(dy, x, m2, r2, w)
        assert torch.isfinite(dx[:4]).all() and torch.isnan(dx[4:]).all() and torch.isnan(dw).all() and torch.isfinite(db).all()


def test_gradients_against_differences():
    """Central differences of the fp64 formula at step 1e-5: its third derivative, of some units, leaves below 1e-9."""
    g = glowq()
    x, w, b, dy = made(4, 24, "f32", 3)
    _, mean, rstd = g.layer_norm(x, w, b, 1e-5)
    dx, dw, db = (R.f64(t) for t in g.layer_norm_backward(dy, x, mean, rstd, w))
    (_, bx), (_, bw), (_, bb) = Q.norm_backward(dy, x, mean, rstd, w, "f32")
    xf, wf, bf, gf = (R.f64(t) for t in (x, w, b, dy))
    eps = float(np.float32(1e-5))

    def loss(xx, ww, bb_):
        c = xx - xx.mean(1, keepdims=True)
        return float((gf * (c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * ww + bb_)).sum())
    # the forward's mean and rstd are rounded: what they move dx and dw by
    slack = 64 * Q.U32 * np.abs(gf).max() * (1 + np.abs(xf).max() * float(rstd.max())) ** 2 * float(rstd.max()) * 24
    for t in range(4):
        for c in range(24):
            up, down = xf.copy(), xf.copy()
            up[t, c] += 1e-5
            down[t, c] -= 1e-5
            assert abs((loss(up, wf, bf) - loss(down, wf, bf)) / 2e-5 - dx[t, c]) <= bx[t, c] + slack + 1e-8
    for c in range(24):
        one = np.eye(24)[c] * 1e-5
        assert abs((loss(xf, wf + one, bf) - loss(xf, wf - one, bf)) / 2e-5 - dw[c]) <= bw[c] + slack + 1e-8
        assert abs((loss(xf, wf, bf + one) - loss(xf, wf, bf - one)) / 2e-5 - db[c]) <= bb[c] + 1e-8


def test_in_place_outputs_streams_and_workspaces():
    g = glowq()
    for shape in ((515, 2048), (33, 250), (5, 16384)):
        x, w, b, dy = made(*shape, "f16", 9)
        y, mean, rstd = g.layer_norm(x, w, b)
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w)
        ws = torch.full((g.layer_norm_workspace_bytes(*shape),), 0xFF, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for into in ("x", "dy"):
            xx, gg = x.clone(), dy.clone()
            torch.cuda.synchronize()
            out = (xx if into == "x" else gg, torch.empty_like(dw), torch.empty_like(db))
            got = g.layer_norm_backward(gg, xx, mean, rstd, w, ws, out, stream=side)
            side.synchronize()
            assert got[0] is out[0] and torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
        xx = x.clone()
        got = g.layer_norm(xx, w, b, out=(xx, torch.empty_like(mean), torch.empty_like(rstd)))
        assert got[0] is xx and torch.equal(xx, y) and torch.equal(got[1], mean)


def test_captured_and_replayed():
    g = glowq()
    x, w, b, dy = made(300, 1000, "f16", 9)
    ws = torch.empty(g.layer_norm_workspace_bytes(300, 1000), dtype=torch.uint8, device="cuda")
    run = lambda k: (lambda f: f + g.layer_norm_backward(dy, x, f[1], f[2], w, k))(g.layer_norm(x, w, b))
    eager = run(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ws)
    for seed in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager))
        x.copy_(made(300, 1000, "f16", 20 + seed)[0])
        eager = run(None)


def test_refusals():
    g = glowq()
    x, w, b, dy = made(8, 64, "f16", 1)
    y, mean, rstd = g.layer_norm(x, w, b)
    big = torch.empty(1, 16385, device="cuda")
    ws = torch.empty(g.layer_norm_workspace_bytes(8, 64), dtype=torch.uint8, device="cuda")
    flat = torch.empty(1024, dtype=torch.float16, device="cuda")
    bad = [lambda: g.layer_norm(x.double()), lambda: g.layer_norm(x[0]), lambda: g.layer_norm(x.t()), lambda: g.layer_norm(x.cpu()),
           lambda: g.layer_norm(x, w.float()), lambda: g.layer_norm(x, w[:63]), lambda: g.layer_norm(x, eps=-1.0),
           lambda: g.layer_norm(x, eps=float("nan")), lambda: g.layer_norm(big), lambda: g.layer_norm(x, out=(y[:7], mean, rstd)),
           lambda: g.layer_norm(x, out=(y, mean, mean)), lambda: g.layer_norm(flat[:512].view(8, 64), out=(flat[8:520].view(8, 64), mean, rstd)),
           lambda: g.layer_norm_backward(dy.float(), x, mean, rstd, w), lambda: g.layer_norm_backward(dy, x, mean[:7], rstd, w),
           lambda: g.layer_norm_backward(dy, x, mean.half(), rstd, w), lambda: g.layer_norm_backward(dy, x, mean, rstd, w, ws[:256]),
           lambda: g.layer_norm_backward(dy, x, mean, rstd, w, ws, (dy, mean[:0], rstd))]
    for i, f in enumerate(bad):
        with pytest.raises(g.GlowQError):
            f()
            print("accepted", i)
