"""The largest batches of the router, the layer norm and the block-scaled FP8 products (2^20 tokens, 2^23 rows over experts): the first, the
last and some rows between against the fp64 references; one token more is refused."""
import pytest
import torch

import fp8_ref as F
import layer_ref as R
import router_ref as Q
from gpu_util import glowq, log

pytestmark = pytest.mark.gpu
T = 1 << 20
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def some(n, seed=0):
    """The ends, both sides of 2^16 and 2^19, and others."""
    gen = torch.Generator().manual_seed(seed)
    return torch.cat([torch.tensor([0, 1, 65535, 65536, (1 << 19) - 1, 1 << 19, n - 2, n - 1]), torch.randint(0, n, (24,), generator=gen)])


@pytest.mark.parametrize("E,k,groups", [(8, 2, 1), (256, 8, 8), (96, 24, 4)])
def test_route(E, k, groups):
    g = glowq()
    gen = torch.Generator("cuda").manual_seed(1)
    lo = torch.randn(T, E, device="cuda", generator=gen)
    bias = 0.1 * torch.randn(E, device="cuda", generator=gen)
    ws = g.init_workspace(torch.empty(8192, dtype=torch.uint8, device="cuda"))
    log(f"route {T} x {E}")
    at = some(T)
    keep = max(1, groups // 2)
    for score, b, renorm in (("softmax", None, False), ("sigmoid", bias, True)):
        ids, w = g.moe_route(lo, k, score, b, groups, keep, 2 if b is not None else 1, renorm, 2.5, ws)
        ri, rw, rb = Q.route(lo[at.cuda()], k, score, None if b is None else b, groups, keep, 2 if b is not None else 1, renorm, 2.5)
        assert (ids[at.cuda()].cpu().numpy() == ri).all()
        R.within(w[at.cuda()], rw, rb, "weights")
        dw = torch.randn(T, k, device="cuda", generator=gen)
        got = g.moe_route_backward(dw, lo, ids, score, renorm, 2.5, ws)
        ref, bound = Q.route_backward(dw[at.cuda()], lo[at.cuda()], ids[at.cuda()], score, renorm, 2.5, "f32")
        R.within(got[at.cuda()], ref, bound, "gradient")
    assert g.workspace_status(ws) == g.OK
    with pytest.raises(g.GlowQError):
        g.moe_route(torch.zeros(T + 1, 2, device="cuda"), 1, workspace=ws)


@pytest.mark.parametrize("kind,d", [("f16", 17), ("f32", 130), ("f16", 1030)])
def test_norm(kind, d):
    g = glowq()
    gen = torch.Generator("cuda").manual_seed(2)
    dt = torch.float16 if kind == "f16" else torch.float32
    x, dy = ((1.0 + torch.randn(T, d, device="cuda", generator=gen)).to(dt) for _ in range(2))
    w, b = (torch.randn(d, device="cuda", generator=gen).to(dt) for _ in range(2))
    log(f"norm {T} x {d} {kind}")
    at = some(T).cuda()
    y, mean, rstd = g.layer_norm(x, w, b)
    for got, (ref, bound), name in zip((y[at], mean[at], rstd[at]), Q.norm(x[at], w, b, 1e-5, kind), ("y", "mean", "rstd")):
        R.within(got, ref, bound, name)
    dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w)
    ref, bound = Q.norm_backward(dy[at], x[at], mean[at], rstd[at], w, kind)[0]
    R.within(dx[at], ref, bound, "dx")
    sums, mags = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)], [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for i in range(0, T, 1 << 16):
        j = slice(i, i + (1 << 16))
        gd = dy[j].double()
        for n, term in enumerate((gd * (x[j].double() - mean[j].double()[:, None]) * rstd[j].double()[:, None], gd)):
            sums[n] += term.sum(0)
            mags[n] += term.abs().sum(0)
    chain = T // 256 + 64 + 16 + 16 + 6  # additions of one value, as router_ref.norm_backward counts them
    for got, s, m, name in zip((dw, db), sums, mags, ("dw", "db")):
        R.within(got, s.cpu().numpy(), chain * Q.U32 * m.cpu().numpy() + 2.0 ** -149, name)
    with pytest.raises(g.GlowQError):
        g.layer_norm(torch.zeros(T + 1, 2, device="cuda"))


def test_fp8_group():
    g = glowq()
    d, n, r = 128, 40, 8
    gen = torch.Generator().manual_seed(3)
    q, s = (100 * torch.randn(n, d, generator=gen)).clamp(-448, 448).to(E4M3), 0.001 * torch.rand(1, 1, generator=gen)
    a, b = (0.3 * torch.randn(n, r, generator=gen)).half(), (torch.randn(r, d, generator=gen) / d ** 0.5).half()
    x = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).half()
    log("fp8 2^20 tokens")
    y = g.group_forward_fp8(x, [g.QWeight.from_fp8(q, s)], b.cuda(), [a.cuda()], r)[0]
    at = some(T)
    R.within(y[at.cuda()], *F.product(x[at.cuda()].cpu(), q, s, b, a, True), "2^20 tokens")
    with pytest.raises(g.GlowQError):
        g.group_forward_fp8(torch.zeros(T + 1, d, dtype=torch.float16, device="cuda"), [g.QWeight.from_fp8(q, s)], None, [], 0, False)


@pytest.mark.parametrize("share", ["expert", "all"])
def test_fp8_experts(share):
    """2^23 rows of 2^20 tokens over 7 experts, through the routing lists."""
    g = glowq()
    d, n, r, E, k = 128, 20, 8, 7, 8
    how = g.MOE_SHARE_EXPERT if share == "expert" else g.MOE_SHARE_ALL
    gen = torch.Generator().manual_seed(5)
    q = [(100 * torch.randn(n, d, generator=gen)).clamp(-448, 448).to(E4M3) for _ in range(E)]
    s = [0.001 * torch.rand(1, 1, generator=gen) for _ in range(E)]
    a = [(0.3 * torch.randn(n, r, generator=gen)).half() for _ in range(E)]
    b = (torch.randn(*((E, r, d) if share == "expert" else (r, d)), generator=gen) / d ** 0.5).half()
    mod = g.MoeModule.stack([g.QWeight.from_fp8(*p) for p in zip(q, s)], [t.cuda() for t in a])
    gpu = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(T, d, device="cuda", generator=gpu).half()
    ids = torch.randint(0, E, (T, k), device="cuda", generator=gpu, dtype=torch.int32)
    off, tok, _ = g.moe_sort(ids, E)
    log(f"fp8 experts 2^23 rows {share}")
    y = g.moe_forward_fp8(x, E, [mod], b.cuda(), how, r, True, tok, off, T * k)[0]
    o = off.tolist()
    for e in range(E):
        at = torch.cat([torch.tensor([o[e], o[e] + 1, o[e + 1] - 2, o[e + 1] - 1]), torch.randint(o[e], o[e + 1], (12,), generator=gen)]).cuda()
        xe = x[tok[at].long()].cpu()
        R.within(y[at], *F.product(xe, q[e], s[e], b[e] if share == "expert" else b, a[e], True), f"expert {e}")
