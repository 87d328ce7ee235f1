"""An MoE layer end to end on the library's calls: routing lists, the INT4 experts' gate/up, the gated
activation, the INT4 down projection, and the weighted way back onto a shared expert computed on 8-bit
integer weights -- each call against its fp64 reference on the tensors the call really had, and the
layer's result against the whole layer in fp64."""
import numpy as np
import pytest
import torch

import layer_ref as R
import workload as W
from gpu_util import assert_parity, glowq, log
from oracle import glowq_ref as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


def int8(w):
    s = w.float().abs().amax(1) / 127.0
    return torch.round(w.float() / s[:, None]).clamp(-127, 127).to(torch.int8), s


@pytest.mark.parametrize("T", [1, 9, 130])
def test_moe_layer(T):
    g = glowq()
    E, k, d, f, r = 6, 2, 256, 384, 16
    x = W.make_x(T, d, 0.77, (90, T)) * 0.5
    units = [W.make_unit(f"e{e}", "group", torch.zeros(1, d).half(), [f, f], r, (91, e)) for e in range(E)]
    downs = [W.make_unit(f"d{e}", "solo", torch.zeros(1, f).half(), [d], r, (92, e)) for e in range(E)]
    mods = [g.MoeModule.stack([g.QWeight.from_workload(u.weights[i]) for u in units], [u.a[i].cuda() for u in units])
            for i in range(2)]
    dmod = [g.MoeModule.stack([g.QWeight.from_workload(u.weights[0]) for u in downs], [u.a[0].cuda() for u in downs])]
    b, bd = torch.stack([u.b.cuda() for u in units]), torch.stack([u.b.cuda() for u in downs])
    gen = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=gen)
    top = torch.topk(torch.softmax(logits, 1), k, 1)
    ids, w = top.indices.to(torch.int32), top.values.float()
    sw = [int8(0.05 * torch.randn(f, d, generator=gen)) for _ in range(2)]
    sd = int8(0.05 * torch.randn(d, f, generator=gen))

    n = T * k
    need = max(g.moe_workspace_bytes(n, T, r, 0), g.moe_workspace_bytes(n, n, r, 0), g.moe_sort_workspace_bytes(T, k, E))
    ws = g.make_workspace(1, 8, 1, min_bytes=need)
    xc, wc = x.cuda(), w.cuda()
    off, tok, pr = g.moe_sort(ids.cuda(), E, workspace=ws)
    gu = g.moe_forward(xc, E, mods, b, g.MOE_SHARE_EXPERT, r, True, tok, off, n, workspace=ws)
    h = g.swiglu(gu[0], gu[1])
    out = g.moe_forward(h, E, dmod, bd, g.MOE_SHARE_EXPERT, r, True, None, off, n, workspace=ws)[0]
    sg = g.group_forward_w8a8(xc, [g.QWeight.from_int8(q, s) for q, s in sw], None, [], 0, False)
    sh = g.swiglu(sg[0], sg[1])
    so = g.group_forward_w8a8(sh, [g.QWeight.from_int8(*sd)], None, [], 0, False)[0]
    y = g.moe_combine(out, pr, wc, add=so, workspace=ws)
    assert g.workspace_status(ws) == g.OK

    # call by call
    ro, rt, rp = R.sort(ids, E)
    for a, c in zip((off, tok, pr), (ro, rt, rp)):
        assert np.array_equal(a.cpu().numpy(), c)
    for got, codes in ((sg, sw), ([so], [sd])):
        ref, bound = R.w8a8(x if got is sg else sh.cpu(), [c[0] for c in codes], [c[1] for c in codes], None, [], False)
        for a, c, bd_ in zip(got, ref, bound):
            R.within(a, c, bd_, "shared expert")
    R.within(h, *R.swiglu(gu[0], gu[1], "f16"), "h")
    R.within(y, *R.combine(out, rp, w.double().numpy(), so, "f16"), "combine")

    # the whole layer in fp64 (the 8-bit codes of the shared expert as the library's: they are exact)
    silu = lambda v: v / (1.0 + np.exp(-v))
    xf = R.f64(x)
    total = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            ge, ue = [xf[t] @ G.dequant_qw(units[e].weights[i]).T + (xf[t] @ R.f64(units[e].b).T) @ R.f64(units[e].a[i]).T
                      for i in range(2)]
            he = silu(ge) * ue
            total[t] += float(w[t, j]) * (he @ G.dequant_qw(downs[e].weights[0]).T +
                                          (he @ R.f64(downs[e].b).T) @ R.f64(downs[e].a[0]).T)
    total += R.w8a8(sh.cpu(), [sd[0]], [sd[1]], None, [], False)[0][0]
    log(f"layer T={T}")
    assert_parity(y, total, f"MoE layer T={T}")
