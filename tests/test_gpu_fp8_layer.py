"""A mixture-of-experts layer on block-scaled e4m3 weights on the library's calls: norm, router, routing lists, the experts' and
a shared expert's products, the gated activation and the weighted way back, and the router's and the norm's gradients -- each
call against its fp64 reference on the tensors the call really had, and the whole captured and replayed."""
import numpy as np
import pytest
import torch

import fp8_ref as F
import layer_ref as R
import router_ref as S
from gpu_util import glowq, log

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


class Proj:
    """One module of one expert: codes, scales, A and (beside it) its B."""

    def __init__(self, n, d, r, gen):
        rn = lambda *s: torch.randn(*s, generator=gen)
        self.q = (100 * rn(n, d)).clamp(-448, 448).to(E4M3)
        self.s = (0.5 + torch.rand(-(-n // 128), d // 128, generator=gen)) * 0.01 / d ** 0.5
        self.a = (0.1 * rn(n, r)).half()

    def weight(self):
        return glowq().QWeight.from_fp8(self.q, self.s)


class Layer:
    def __init__(self, T, E, k, d, f, r, seed):
        g = glowq()
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)
        self.T, self.E, self.k, self.d, self.f, self.r = T, E, k, d, f, r
        self.x = (rn(T, d) * (0.3 + rn(1, d).abs())).half()
        self.nw, self.nb = (1 + 0.1 * rn(d)).half(), (0.1 * rn(d)).half()
        self.wg = rn(E, d) / d ** 0.5
        self.bias = 0.05 * rn(E)
        self.up = [[Proj(f, d, r, gen) for _ in range(E + 1)] for _ in range(2)]   # the last: the shared expert
        self.down = [Proj(d, f, r, gen) for _ in range(E + 1)]
        self.b1, self.b2 = (rn(E + 1, r, d) / d ** 0.5).half(), (rn(E + 1, r, f) / f ** 0.5).half()
        stack = lambda p: g.MoeModule.stack([u.weight() for u in p[:E]], [u.a.cuda() for u in p[:E]])
        self.mods, self.dmod = [stack(p) for p in self.up], [stack(self.down)]
        self.sw, self.sd = [p[E].weight() for p in self.up], [self.down[E].weight()]
        self.sa, self.sda = [p[E].a.cuda() for p in self.up], [self.down[E].a.cuda()]
        n, most = T * k, max(d, f)
        need = max(g.moe_fp8_workspace_bytes(n, T, d, r, 0), g.moe_fp8_workspace_bytes(n, n, f, r, 0), g.moe_sort_workspace_bytes(T, k, E))
        self.ws = g.init_workspace(torch.empty(need, dtype=torch.uint8, device="cuda"))
        self.ws2 = torch.empty(g.fp8_workspace_bytes(T, most, r), dtype=torch.uint8, device="cuda")
        self.dev = {n: getattr(self, n).cuda() for n in ("nw", "nb", "wg", "bias", "b1", "b2")}

    def forward(self, x):
        g, c, n = glowq(), self.dev, self.T * self.k
        y = {}
        y["norm"] = g.layer_norm(x, c["nw"], c["nb"])
        h = y["norm"][0]
        y["logits"] = h.float() @ c["wg"].t()
        y["route"] = g.moe_route(y["logits"], self.k, "sigmoid", c["bias"], n_group=4, keep_groups=2, group_best=2, scale=1.5, workspace=self.ws)
        y["lists"] = g.moe_sort(y["route"][0], self.E, workspace=self.ws)
        off, tok, pr = y["lists"]
        y["gu"] = g.moe_forward_fp8(h, self.E, self.mods, c["b1"][:self.E], g.MOE_SHARE_EXPERT, self.r, True, tok, off, n, workspace=self.ws)
        y["act"] = g.swiglu(*y["gu"])
        y["rows"] = g.moe_forward_fp8(y["act"], self.E, self.dmod, c["b2"][:self.E], g.MOE_SHARE_EXPERT, self.r, True, None, off, n,
                                      workspace=self.ws)[0]
        y["sgu"] = g.group_forward_fp8(h, self.sw, c["b1"][self.E], self.sa, self.r, workspace=self.ws2)
        y["sact"] = g.swiglu(*y["sgu"])
        y["shared"] = g.group_forward_fp8(y["sact"], self.sd, c["b2"][self.E], self.sda, self.r, workspace=self.ws2)[0]
        y["out"] = g.moe_combine(y["rows"], pr, y["route"][1], add=y["shared"], workspace=self.ws)
        return y

    def backward(self, dy, x, y):
        """Of the router's weights down to x (through the router's product)."""
        g, c = glowq(), self.dev
        off, tok, pr = y["lists"]
        d_rows, d_w = g.moe_combine_backward(dy, y["rows"], pr, tok, y["route"][1], workspace=self.ws)
        d_logits = g.moe_route_backward(d_w, y["logits"], y["route"][0], "sigmoid", scale=1.5, workspace=self.ws)
        dh = (d_logits @ c["wg"]).half()
        return d_rows, d_w, d_logits, dh, g.layer_norm_backward(dh, x, y["norm"][1], y["norm"][2], c["nw"])


SHAPES = [(1, 8, 2, 256, 384, 8), (9, 8, 2, 256, 384, 16), (150, 8, 3, 384, 256, 64), (70, 48, 4, 128, 640, 24)]


@pytest.mark.parametrize("T,E,k,d,f,r", SHAPES)
def test_layer_call_by_call(T, E, k, d, f, r):
    g = glowq()
    u = Layer(T, E, k, d, f, r, T)
    x = u.x.cuda()
    log(f"fp8 layer T={T} E={E} k={k} d={d} f={f} r={r}")
    y = u.forward(x)
    assert g.workspace_status(u.ws) == g.OK
    (h, hb), (mean, mb), (rstd, rb) = S.norm(u.x, u.nw, u.nb, 1e-5, "f16")
    for got, ref, bound, what in zip(y["norm"], (h, mean, rstd), (hb, mb, rb), ("norm", "mean", "rstd")):
        R.within(got, ref, bound, what)
    ids, w, wb = S.route(y["logits"], k, "sigmoid", u.bias, 4, 2, 2, True, 1.5)
    assert np.array_equal(y["route"][0].cpu().numpy(), ids)
    R.within(y["route"][1], w, wb, "weights")
    lists = R.sort(y["route"][0].cpu(), E)
    for got, ref in zip(y["lists"], lists):
        assert np.array_equal(got.cpu().numpy(), ref)
    off, tok, pr = lists
    hx = y["norm"][0].cpu()
    for e in range(E):
        j = slice(off[e], off[e + 1])
        if j.start == j.stop:
            continue
        for i in range(2):
            p = u.up[i][e]
            R.within(y["gu"][i][j], *F.product(hx[tok[j].astype(np.int64)], p.q, p.s, u.b1[e], p.a, True), f"expert {e}")
        p = u.down[e]
        R.within(y["rows"][j], *F.product(y["act"][j], p.q, p.s, u.b2[e], p.a, True), f"expert {e} down")
    R.within(y["act"], *R.swiglu(*y["gu"], "f16"), "act")
    for i in range(2):
        p = u.up[i][E]
        R.within(y["sgu"][i], *F.product(hx, p.q, p.s, u.b1[E], p.a, True), "shared")
    p = u.down[E]
    R.within(y["shared"], *F.product(y["sact"], p.q, p.s, u.b2[E], p.a, True), "shared down")
    R.within(y["out"], *R.combine(y["rows"], pr, R.f64(y["route"][1]), y["shared"], "f16"), "out")

    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(3)).half()
    d_rows, d_w, d_logits, dh, (dx, dnw, dnb) = u.backward(dy.cuda(), x, y)
    dr, drb, dw, dwb, _ = R.combine_backward(dy, y["rows"], pr, R.f64(y["route"][1]), T * k, "f16")
    R.within(d_rows, dr, drb, "d_rows")
    R.within(d_w, dw, dwb, "d_weights")
    R.within(d_logits, *S.route_backward(d_w, y["logits"], y["route"][0], "sigmoid", True, 1.5, "f32"), "d_logits")
    ref = S.norm_backward(dh, u.x, y["norm"][1], y["norm"][2], u.nw, "f16")
    for got, (v, bound), what in zip((dx, dnw, dnb), ref, ("dx", "d_weight", "d_bias")):
        R.within(got, v, bound, what)


@pytest.mark.parametrize("T,E,k,d,f,r", SHAPES[1:])
def test_layer_captured_and_replayed(T, E, k, d, f, r):
    """Forward calls in one graph, replayed on new inputs with eager calls between."""
    g = glowq()
    u = Layer(T, E, k, d, f, r, 7)
    x = u.x.cuda()
    eager = u.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = u.forward(x)
    for seed in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held["route"][0], eager["route"][0]) and torch.equal(held["out"], eager["out"])
        x.copy_(torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).half())
        eager = u.forward(x)
    assert g.workspace_status(u.ws) == g.OK
