"""The router's and the layer norm's calls without a GPU: sizes, and every refusal before any HIP call."""
import ctypes

import pytest

from rank_error_compensation_amd import glowq as g

FAKE = 0x10000   # aligned fake device address: never dereferenced, validation fails first
FAR = 0x40000000
HDR = 8192


def route(x=FAKE, T=4, E=60, k=4, dtype=1, score=0, bias=None, G=1, keep=1, best=1, renorm=1, scale=1.0, ids=FAR, w=2 * FAR,
          ws=3 * FAR, n=HDR):
    return g.lib().glowq_moe_route(x, T, E, k, dtype, score, bias, G, keep, best, renorm, scale, ids, w, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), g.ERR_INVALID_ARG), (dict(ids=None), g.ERR_INVALID_ARG), (dict(w=None), g.ERR_INVALID_ARG),
    (dict(dtype=2), g.ERR_INVALID_ARG), (dict(score=2), g.ERR_INVALID_ARG), (dict(score=-1), g.ERR_INVALID_ARG),
    (dict(best=0), g.ERR_INVALID_ARG), (dict(best=3), g.ERR_INVALID_ARG), (dict(scale=float("nan")), g.ERR_INVALID_ARG),
    (dict(scale=float("-inf")), g.ERR_INVALID_ARG), (dict(T=-1), g.ERR_SHAPE), (dict(E=0), g.ERR_SHAPE), (dict(k=0), g.ERR_SHAPE),
    (dict(k=61), g.ERR_SHAPE), (dict(G=7), g.ERR_SHAPE), (dict(G=0), g.ERR_SHAPE), (dict(G=4, keep=5), g.ERR_SHAPE),
    (dict(G=4, keep=0), g.ERR_SHAPE), (dict(E=64, G=32, keep=4), g.ERR_UNSUPPORTED), (dict(E=257), g.ERR_UNSUPPORTED),
    (dict(E=256, k=65), g.ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), g.ERR_UNSUPPORTED), (dict(x=FAKE + 8), g.ERR_ALIGN),
    (dict(bias=FAKE + 2), g.ERR_ALIGN), (dict(ids=FAR + 2), g.ERR_ALIGN), (dict(w=FAR + 2), g.ERR_ALIGN),
    (dict(ws=None), g.ERR_WORKSPACE), (dict(n=HDR - 1), g.ERR_WORKSPACE), (dict(ws=FAR * 3 + 128), g.ERR_ALIGN),
    (dict(w=FAR + 60), g.ERR_INVALID_ARG), (dict(ids=FAKE + 476), g.ERR_INVALID_ARG), (dict(w=FAKE), g.ERR_INVALID_ARG),
    (dict(bias=FAR), g.ERR_INVALID_ARG), (dict(T=0, x=None), g.OK),
])
def test_route_refusals(kw, status):
    assert route(**kw) == status


def route_back(dw=FAKE, x=FAR, ids=2 * FAR, T=4, E=60, k=4, dtype=1, score=1, renorm=1, scale=1.0, out=3 * FAR, ws=4 * FAR, n=HDR):
    return g.lib().glowq_moe_route_backward(dw, x, ids, T, E, k, dtype, score, renorm, scale, out, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dw=None), g.ERR_INVALID_ARG), (dict(x=None), g.ERR_INVALID_ARG), (dict(ids=None), g.ERR_INVALID_ARG),
    (dict(out=None), g.ERR_INVALID_ARG), (dict(dtype=5), g.ERR_INVALID_ARG), (dict(score=7), g.ERR_INVALID_ARG),
    (dict(scale=float("inf")), g.ERR_INVALID_ARG), (dict(T=-1), g.ERR_SHAPE), (dict(E=0), g.ERR_SHAPE), (dict(k=0), g.ERR_SHAPE),
    (dict(k=65), g.ERR_UNSUPPORTED), (dict(E=300), g.ERR_UNSUPPORTED), (dict(T=1 << 21), g.ERR_UNSUPPORTED),
    (dict(x=FAR + 8), g.ERR_ALIGN), (dict(out=FAR * 3 + 8), g.ERR_ALIGN), (dict(dw=FAKE + 2), g.ERR_ALIGN),
    (dict(ids=FAR + 1), g.ERR_ALIGN), (dict(out=FAR + 16), g.ERR_INVALID_ARG), (dict(out=FAKE - 464), g.ERR_INVALID_ARG),
    (dict(out=2 * FAR), g.ERR_INVALID_ARG), (dict(ws=None), g.ERR_WORKSPACE), (dict(n=100), g.ERR_WORKSPACE), (dict(T=0), g.OK),
])
def test_route_backward_refusals(kw, status):
    assert route_back(**kw) == status


def norm(x=FAKE, w=FAR, b=2 * FAR, T=4, d=64, eps=1e-5, dtype=1, y=3 * FAR, mean=4 * FAR, rstd=5 * FAR):
    return g.lib().glowq_layer_norm(x, w, b, T, d, eps, dtype, y, mean, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), g.ERR_INVALID_ARG), (dict(y=None), g.ERR_INVALID_ARG), (dict(dtype=2), g.ERR_INVALID_ARG),
    (dict(eps=-1e-5), g.ERR_INVALID_ARG), (dict(eps=float("inf")), g.ERR_INVALID_ARG), (dict(eps=float("nan")), g.ERR_INVALID_ARG),
    (dict(T=-1), g.ERR_SHAPE), (dict(d=0), g.ERR_SHAPE), (dict(d=16385), g.ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), g.ERR_UNSUPPORTED),
    (dict(x=FAKE + 4), g.ERR_ALIGN), (dict(w=FAR + 2), g.ERR_ALIGN), (dict(b=FAR + 2), g.ERR_ALIGN), (dict(y=FAR * 3 + 2), g.ERR_ALIGN),
    (dict(mean=FAR * 4 + 2), g.ERR_ALIGN), (dict(rstd=FAR * 4 + 2), g.ERR_ALIGN), (dict(y=FAKE + 16), g.ERR_INVALID_ARG),
    (dict(y=FAR + 112), g.ERR_INVALID_ARG), (dict(mean=5 * FAR + 12), g.ERR_INVALID_ARG), (dict(mean=FAKE + 508), g.ERR_INVALID_ARG),
    (dict(rstd=3 * FAR), g.ERR_INVALID_ARG), (dict(rstd=FAR), g.ERR_INVALID_ARG), (dict(T=0, x=None), g.OK),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def norm_back(dy=FAKE, x=FAR, mean=2 * FAR, rstd=3 * FAR, w=4 * FAR, T=4, d=64, dtype=0, dx=5 * FAR, dw=6 * FAR, db=7 * FAR,
              ws=8 * FAR, n=1 << 30):
    return g.lib().glowq_layer_norm_backward(dy, x, mean, rstd, w, T, d, dtype, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), g.ERR_INVALID_ARG), (dict(x=None), g.ERR_INVALID_ARG), (dict(mean=None), g.ERR_INVALID_ARG),
    (dict(rstd=None), g.ERR_INVALID_ARG), (dict(dx=None), g.ERR_INVALID_ARG), (dict(dtype=3), g.ERR_INVALID_ARG),
    (dict(T=-2), g.ERR_SHAPE), (dict(d=-1), g.ERR_SHAPE), (dict(d=20000), g.ERR_UNSUPPORTED), (dict(T=1 << 21), g.ERR_UNSUPPORTED),
    (dict(dy=FAKE + 4), g.ERR_ALIGN), (dict(x=FAR + 4), g.ERR_ALIGN), (dict(dx=FAR * 5 + 4), g.ERR_ALIGN), (dict(w=FAR * 4 + 8), g.ERR_ALIGN),
    (dict(dw=FAR * 6 + 2), g.ERR_ALIGN), (dict(db=FAR * 6 + 2), g.ERR_ALIGN), (dict(mean=FAR * 2 + 1), g.ERR_ALIGN),
    (dict(ws=None), g.ERR_WORKSPACE), (dict(n=256), g.ERR_WORKSPACE), (dict(ws=FAR * 8 + 64), g.ERR_ALIGN),
    (dict(dx=FAKE + 32), g.ERR_INVALID_ARG), (dict(dx=FAR + 32), g.ERR_INVALID_ARG), (dict(dx=4 * FAR), g.ERR_INVALID_ARG),
    (dict(dx=2 * FAR), g.ERR_INVALID_ARG), (dict(dw=7 * FAR + 4), g.ERR_INVALID_ARG), (dict(dw=5 * FAR), g.ERR_INVALID_ARG),
    (dict(db=FAKE), g.ERR_INVALID_ARG), (dict(db=3 * FAR), g.ERR_INVALID_ARG), (dict(T=0, dw=None, db=None, ws=None), g.OK),
])
def test_norm_backward_refusals(kw, status):
    assert norm_back(**kw) == status


def test_norm_workspace_bytes():
    f = g.lib().glowq_layer_norm_workspace_bytes
    assert f(0, 1) >= 8 and f(4096, 4096) >= 2 * 4096 * 4
    for T, d in ((-1, 64), ((1 << 20) + 1, 64), (4, 0), (4, 16385)):
        assert f(T, d) == 0
    assert [f(T, 512) for T in (1, 100, 5000)] == sorted(f(T, 512) for T in (1, 100, 5000))
