"""The router (glowq_moe_route and its gradient) against the definition in fp64: equal ids, weights and
gradients within the bounds of their roundings."""
import math

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


def ws():
    g = glowq()
    return g.init_workspace(torch.empty(8192, dtype=torch.uint8, device="cuda"))


def made(T, E, kind, seed, masked=False):
    gen = torch.Generator().manual_seed(seed)
    lo = (1.5 * torch.randn(T, E, generator=gen) + 0.7 * torch.randn(1, E, generator=gen)).to(KINDS[kind])
    if masked:
        lo[torch.rand(T, E, generator=gen) < 0.3] = -math.inf
        lo[torch.rand(T, generator=gen) < 0.2] = -math.inf
        if T > 1:
            lo[1] = -math.inf
            lo[1, E - 1] = 0.5  # one expert left
    return lo, 0.1 * torch.randn(E, generator=gen)


def check(lo, k, score="softmax", bias=None, n_group=1, keep=1, best=1, renorm=True, scale=1.0, what=""):
    g = glowq()
    w_ = ws()
    ids, w = g.moe_route(lo.cuda(), k, score, None if bias is None else bias.cuda(), n_group, keep, best, renorm, scale, w_)
    ri, rw, rb = Q.route(lo, k, score, bias, n_group, keep, best, renorm, scale)
    diff = np.argwhere(ids.cpu().numpy() != ri)
    assert diff.size == 0, (what, diff[:4].tolist(), ids[diff[0][0]].tolist(), ri[diff[0][0]].tolist())
    R.within(w, rw, rb, f"{what} weights")
    assert g.workspace_status(w_) == g.OK
    return ids, w


# (T, experts, top_k, groups, kept groups): one expert, sizes around the lists' and lanes' limits, every kernel
SIZES = [(1, 1, 1, 1, 1), (1, 60, 4, 1, 1), (3, 2, 2, 1, 1), (17, 64, 8, 8, 3), (33, 65, 4, 5, 2), (16, 100, 8, 4, 4),
         (50, 128, 1, 16, 16), (31, 128, 8, 16, 4), (65, 129, 3, 3, 1), (40, 256, 8, 8, 4), (29, 256, 4, 2, 1), (37, 255, 5, 15, 7),
         (21, 64, 64, 1, 1), (9, 256, 64, 4, 2), (30, 30, 9, 2, 1), (13, 200, 16, 8, 8), (5, 16, 16, 16, 16), (130, 12, 3, 4, 2)]


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_choice_and_weights(size, kind):
    T, E, k, G, keep = size
    for n, (score, biased, best, renorm) in enumerate([("softmax", False, 1, True), ("softmax", False, 2, False),
                                                       ("sigmoid", True, 2, True), ("sigmoid", False, 1, False),
                                                       ("softmax", True, 1, True), ("sigmoid", True, 1, False)]):
        for masked in (False, True):
            log(f"route {size} {kind} {score} bias={biased} best={best} renorm={renorm} masked={masked}")
            lo, b = made(T, E, kind, 100 * n + masked, masked)
            check(lo, k, score, b if biased else None, G, keep, best, renorm, 2.5 if n % 2 else 1.0, f"{score} {n}")


@pytest.mark.parametrize("k,E", [(4, 60), (8, 256), (20, 128)])
def test_equal_values_go_to_the_lower_expert(k, E):
    """Whole-number logits: many ties, also between 0 and -0."""
    gen = torch.Generator().manual_seed(5)
    lo = torch.randint(-2, 3, (64, E), generator=gen).float()
    lo[lo == 0] *= torch.where(torch.rand(int((lo == 0).sum()), generator=gen) < 0.5, -1.0, 1.0)
    for kind in ("f16", "f32"):
        check(lo.to(KINDS[kind]), k, what="ties")
        check(lo.to(KINDS[kind]), k, "sigmoid", torch.zeros(E), what="ties with a bias of zeros")
        check(lo.to(KINDS[kind]), min(k, 8), "sigmoid", torch.zeros(E), 4, 2, 2, what="ties in groups")
        check(lo.to(KINDS[kind]), min(k, 8), "softmax", None, 4, 2, 1, what="ties in groups by the best")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(60, 4), (128, 8), (256, 8), (256, 16)])
def test_values_closer_than_fp32_tells_apart(E, k, score):
    """A bias that puts every score within a few fp32 steps of one value: fp64 has to decide."""
    gen = torch.Generator().manual_seed(9)
    lo = torch.randn(1, E, generator=gen).expand(48, E).contiguous()
    s = torch.from_numpy(Q.scores(lo[0].double().numpy(), score))
    bias = (0.75 - s).float()
    lo = lo + 1e-6 * torch.randn(48, E, generator=gen)
    check(lo, k, score, bias, what="close")
    check(lo, k, score, bias, 4, 2, 2, what="close groups")
    check(lo, k, score, None, 4, 2, 2, what="groups by two scores")


def test_ends_of_the_scores():
    """Logits where exp overflows, sigmoids vanish or are 1, subnormal logits; -inf in the bias."""
    base = [0.0, 1e-40, -1e-40, 88.0, -88.0, 100.0, -100.0, 3e38, -3e38, 65504.0, -65504.0, 40.0, 40.5, -200.0, -200.5, 1.0]
    lo = torch.tensor([base, base[::-1], [v * 0.5 for v in base], [-200.0 - i for i in range(16)], [1e4 + i for i in range(16)]])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(lo, 4, score, renorm=renorm, what=f"{score} ends")
            bias = torch.linspace(-1, 1, 16)
            bias[3] = bias[9] = -math.inf
            check(lo, 6, score, bias, renorm=renorm, what=f"{score} ends with a bias")
            check(lo, 16, score, bias, renorm=renorm, what=f"{score} ends, all")


def test_rows_with_nan_or_infinity_are_reported():
    g = glowq()
    lo = torch.randn(6, 60, generator=torch.Generator().manual_seed(1))
    good, _ = check(lo, 4)
    lo[2, 7], lo[4, 59] = float("nan"), math.inf
    w_ = ws()
    ids, w = g.moe_route(lo.cuda(), 4, workspace=w_)
    assert g.workspace_status(w_) == g.ERR_ROUTING and g.workspace_status(w_) == g.OK
    for t in (2, 4):
        assert (ids[t] == -1).all() and (w[t] == 0).all()
    for t in (0, 1, 3, 5):
        assert torch.equal(ids[t], good[t])
    with pytest.raises(g.GlowQError):
        g.moe_route(lo.cuda(), 4)
    bias = torch.zeros(60)
    bias[5] = float("nan")
    ids, w = g.moe_route(lo.cuda(), 4, bias=bias.cuda(), workspace=w_)
    assert (ids == -1).all() and (w == 0).all() and g.workspace_status(w_) == g.ERR_ROUTING


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 60, 4), (17, 64, 8), (33, 65, 16), (40, 256, 8), (16, 128, 1), (9, 200, 64),
                                  (21, 30, 17), (300, 60, 4)], ids=lambda s: "x".join(map(str, s)))
def test_gradient(size, kind):
    g = glowq()
    T, E, k = size
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for masked in (False, True):
                log(f"route gradient {size} {kind} {score} renorm={renorm} masked={masked}")
                lo, _ = made(T, E, kind, 7 + masked, masked)
                w_ = ws()
                ids, _ = g.moe_route(lo.cuda(), min(k, E), score, workspace=w_)
                dw = torch.randn(T, min(k, E), generator=torch.Generator().manual_seed(3))
                got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids, score, renorm, 2.5, w_)
                ref, bound = Q.route_backward(dw, lo, ids, score, renorm, 2.5, kind)
                R.within(got, ref, bound, f"{score} renorm={renorm}")
                assert g.workspace_status(w_) == g.OK


def test_gradient_of_odd_choices():
    """The same expert twice, an expert that is out, ids out of range (reported), more choices than experts."""
    g = glowq()
    lo, _ = made(4, 12, "f32", 1)
    lo[1, 3] = -math.inf
    ids = torch.tensor([[2, 2, 2, 5], [3, 1, 3, 0], [-1, -1, -1, -1], [0, 1, 2, 3]], dtype=torch.int32)
    dw = torch.randn(4, 4, generator=torch.Generator().manual_seed(2))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            w_ = ws()
            got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids.cuda(), score, renorm, 1.5, w_)
            ref, bound = Q.route_backward(dw, lo, ids, score, renorm, 1.5, "f32")
            R.within(got, ref, bound, f"{score} renorm={renorm}")
            assert g.workspace_status(w_) == g.OK
            bad = ids.clone()
            bad[3, 0], bad[3, 1] = 12, -2
            got = g.moe_route_backward(dw.cuda(), lo.cuda(), bad.cuda(), score, renorm, 1.5, w_)
            assert g.workspace_status(w_) == g.ERR_ROUTING
            ref, bound = Q.route_backward(dw, lo, bad, score, renorm, 1.5, "f32")
            R.within(got, ref, bound, "out of range")
    lo, _ = made(5, 3, "f32", 1)
    ids = torch.randint(0, 3, (5, 20), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    dw = torch.randn(5, 20, generator=torch.Generator().manual_seed(2))
    got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids.cuda(), "softmax", True, 1.0, ws())
    ref, bound = Q.route_backward(dw, lo, ids, "softmax", True, 1.0, "f32")
    R.within(got, ref, bound, "20 choices of 3")


def test_gradient_against_differences():
    """Central differences of the fp64 weights at step 1e-5 (third derivatives of these functions are below 1 in
    size, scale 2: below 1e-10 off; the quotient of differences rounds by 1e-11)."""
    g = glowq()
    lo, _ = made(6, 20, "f32", 11)
    dw = torch.randn(6, 4, generator=torch.Generator().manual_seed(2))
    ids, _ = g.moe_route(lo.cuda(), 4)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = R.f64(g.moe_route_backward(dw.cuda(), lo.cuda(), ids, score, renorm, 2.0))
            _, bound = Q.route_backward(dw, lo, ids, score, renorm, 2.0, "f32")
            base, ii, dd = R.f64(lo), ids.cpu().numpy(), R.f64(dw)
            for t in range(6):
                for e in range(20):
                    up, down = base[t].copy(), base[t].copy()
                    up[e] += 1e-5
                    down[e] -= 1e-5
                    num = (Q.weights(up, ii[t], score, renorm, 2.0) - Q.weights(down, ii[t], score, renorm, 2.0)) @ dd[t] / 2e-5
                    assert abs(num - got[t, e]) <= bound[t, e] + 1e-9, (score, renorm, t, e, num, got[t, e])


def test_in_place_out_streams_and_odd_rows():
    g = glowq()
    lo, b = made(33, 61, "f16", 3)
    ids, w = check(lo, 4, "sigmoid", b)
    side = torch.cuda.Stream()
    dev, bias, w_ = lo.cuda(), b.cuda(), ws()
    out = (torch.full((33, 4), 77, dtype=torch.int32, device="cuda"), torch.full((33, 4), 7.0, device="cuda"))
    torch.cuda.synchronize()
    i2, w2 = g.moe_route(dev, 4, "sigmoid", bias, workspace=w_, out=out, stream=side)
    side.synchronize()
    assert i2 is out[0] and torch.equal(i2, ids) and torch.equal(w2, w)
    dw = torch.randn(33, 4, device="cuda")
    a = g.moe_route_backward(dw, dev, ids, "softmax", False, 1.0, w_)
    c = g.moe_route_backward(dw, dev, ids, "softmax", False, 1.0, w_, out=dev)
    assert c is dev and torch.equal(a, c)
    assert g.moe_route(lo[:0].cuda(), 4)[0].shape == (0, 4)


def test_captured_and_replayed():
    g = glowq()
    lo, b = made(300, 256, "f32", 3, masked=True)
    dev, bias, w_ = lo.cuda(), b.cuda(), ws()
    kw = dict(score="sigmoid", bias=bias, n_group=8, keep_groups=4, group_best=2, workspace=w_)
    dw = torch.randn(300, 8, device="cuda")
    eager = g.moe_route(dev, 8, **kw)
    back = g.moe_route_backward(dw, dev, eager[0], "sigmoid", True, 1.0, w_)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = g.moe_route(dev, 8, **kw)
        d = g.moe_route_backward(dw, dev, ids, "sigmoid", True, 1.0, w_)
    for seed in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, eager[0]) and torch.equal(w, eager[1]) and torch.equal(d, back)
        dev.copy_(made(300, 256, "f32", 40 + seed, masked=True)[0])
        eager = g.moe_route(dev, 8, **kw)
        back = g.moe_route_backward(dw, dev, eager[0], "sigmoid", True, 1.0, w_)
    with pytest.raises(g.GlowQError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            g.moe_route(dev, 8)


def test_refusals():
    g = glowq()
    lo = torch.randn(4, 60, device="cuda")
    w_ = ws()
    bad = [lambda: g.moe_route(lo, 0, workspace=w_), lambda: g.moe_route(lo, 61, workspace=w_),
           lambda: g.moe_route(lo, 4, "tanh", workspace=w_), lambda: g.moe_route(lo.double(), 4, workspace=w_),
           lambda: g.moe_route(lo[0], 4, workspace=w_), lambda: g.moe_route(lo.t(), 4, workspace=w_),
           lambda: g.moe_route(lo.cpu(), 4, workspace=w_), lambda: g.moe_route(lo, 4, bias=torch.zeros(59, device="cuda"), workspace=w_),
           lambda: g.moe_route(lo, 4, bias=torch.zeros(60, device="cuda").half(), workspace=w_),
           lambda: g.moe_route(lo, 4, n_group=7, workspace=w_), lambda: g.moe_route(lo, 4, n_group=6, keep_groups=7, workspace=w_),
           lambda: g.moe_route(lo, 4, n_group=6, keep_groups=0, workspace=w_), lambda: g.moe_route(lo, 4, n_group=30, keep_groups=3, workspace=w_),
           lambda: g.moe_route(lo, 4, group_best=3, workspace=w_), lambda: g.moe_route(lo, 4, scale=math.inf, workspace=w_),
           lambda: g.moe_route(lo, 4, workspace=w_[:4096]),
           lambda: g.moe_route_backward(torch.zeros(4, 4, device="cuda"), lo, torch.zeros(4, 5, dtype=torch.int32, device="cuda"), workspace=w_),
           lambda: g.moe_route_backward(torch.zeros(3, 4, device="cuda"), lo, torch.zeros(3, 4, dtype=torch.int32, device="cuda"), workspace=w_),
           lambda: g.moe_route_backward(torch.zeros(4, 4, device="cuda"), lo, torch.zeros(4, 4, dtype=torch.int64, device="cuda"), workspace=w_)]
    for f in bad:
        with pytest.raises(g.GlowQError):
            f()
    assert g.workspace_status(w_) == g.OK
