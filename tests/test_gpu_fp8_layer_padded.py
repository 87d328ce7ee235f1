"""A padded batch through the norm, the router, the experts on block-scaled FP8 weights and back: padding tokens have logits of
-inf alone, the products take the rows that the lists hold."""
import math

import numpy as np
import pytest
import torch

import fp8_ref as F
import layer_ref as R
import router_ref as S
from gpu_util import glowq, log
from test_gpu_moe_fp8 import Layer as Experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,pad,E,k,d,n,r", [(5, [1, 4], 8, 2, 256, 40, 8), (3, [0, 1, 2], 8, 2, 128, 20, 0), (130, range(100, 130), 6, 3, 256, 300, 16)])
def test_padded_batch(T, pad, E, k, d, n, r, score, renorm):
    g = glowq()
    pad = list(pad)
    live = [t for t in range(T) if t not in pad]
    log(f"fp8 padded layer T={T} pad={len(pad)} E={E} {score} renorm={renorm}")
    gen = torch.Generator().manual_seed(T)
    u = Experts(T, d, [n], [1] * E, r, g.MOE_SHARE_EXPERT, T)  # weights; the lists come from the router
    ws = g.init_workspace(torch.empty(max(g.moe_fp8_workspace_bytes(T * k, T, d, r, u.share), g.moe_sort_workspace_bytes(T, k, E)),
                                      dtype=torch.uint8, device="cuda"))
    x, wg = u.x.cuda(), torch.randn(E, d, generator=gen).cuda()
    h, mean, rstd = g.layer_norm(x)
    lo = h.float() @ wg.t() / d ** 0.5
    lo[pad] = -math.inf
    ids, w = g.moe_route(lo, k, score, renorm=renorm, workspace=ws)
    assert (ids[pad] == -1).all() and (w[pad] == 0).all() and (ids[live] >= 0).all()
    off, tok, pr = g.moe_sort(ids, E, workspace=ws)
    rows = int(off[-1])
    assert rows == len(live) * k and (pr[pad] == -1).all()
    y = g.moe_forward_fp8(h, E, u.mods, u.b.cuda() if r else None, u.share, r, True, tok, off, rows, workspace=ws)[0]
    o = off.tolist()
    hc, tc = h.cpu(), tok.cpu().long()
    for e in range(E):
        if o[e] < o[e + 1]:
            R.within(y[o[e]:o[e + 1]], *F.product(hc[tc[o[e]:o[e + 1]]], u.q[0][e], u.s[0][e], u.b[e], u.a[0][e], r > 0), f"expert {e}")
    out = g.moe_combine(y, pr, w, workspace=ws)
    assert (out[pad] == 0).all()
    dy = torch.randn(T, n, generator=gen).half().cuda()
    d_rows, d_w = g.moe_combine_backward(dy, y, pr, tok[:rows], w, workspace=ws)
    assert (d_w[pad] == 0).all()
    d_lo = g.moe_route_backward(d_w, lo, ids, score, renorm, 1.0, ws)
    assert (d_lo[pad] == 0).all()
    R.within(d_lo, *S.route_backward(d_w, lo, ids, score, renorm, 1.0, "f32"), "d_logits")
    dh = (d_lo @ wg / d ** 0.5).half()
    dx, dnw, dnb = g.layer_norm_backward(dh, x, mean, rstd)
    assert (dx[pad] == 0).all()
    for got, (v, bound), what in zip((dx, dnw, dnb), S.norm_backward(dh, x, mean, rstd, None, "f16"), ("dx", "d_weight", "d_bias")):
        R.within(got, v, bound, what)
    assert g.workspace_status(ws) == g.OK
