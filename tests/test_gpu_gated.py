"""Gated activation and its gradients against plain fp64 references and differences."""
import pytest
import torch

import layer_ref as R
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


def values(shape, kind, seed, scale=3.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(KINDS[kind]).cuda()


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("shape", [(1,), (3,), (8,), (9,), (4, 1408), (127, 33), (2, 3, 5, 7), (1000, 1001),
                                   (5003, 4001)])
def test_swiglu_and_gradients(shape, kind):
    g = glowq()
    log(f"swiglu {shape} {kind}")
    gate, up, dh = (values(shape, kind, i) for i in range(3))
    h, b = R.swiglu(gate, up, kind)
    R.within(g.swiglu(gate, up), h, b, "h")
    (dg, bg), (du, bu) = R.swiglu_backward(dh, gate, up, kind)
    a, c = g.swiglu_backward(dh, gate, up)
    R.within(a, dg, bg, "d_gate")
    R.within(c, du, bu, "d_up")


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_far_gates(kind):
    """Both ends of the sigmoid: no overflow, no loss where 1 - s is small."""
    g = glowq()
    ends = [0.0, -0.0, 1e-7, -1e-7, -1.2785, 10.0, -10.0, 17.0, -17.0, 40.0, -40.0, 88.0, -88.0, 100.0, -100.0, 6e4, -6e4]
    gate = torch.tensor(ends).to(KINDS[kind]).cuda()
    up, dh = torch.full_like(gate, 0.5), torch.full_like(gate, 2.0)
    R.within(g.swiglu(gate, up), *R.swiglu(gate, up, kind), "h")
    (dg, bg), (du, bu) = R.swiglu_backward(dh, gate, up, kind)
    a, c = g.swiglu_backward(dh, gate, up)
    R.within(a, dg, bg, "d_gate")
    R.within(c, du, bu, "d_up")
    bad = torch.tensor([float("nan"), 1.0, 1.0, 2.0]).to(KINDS[kind]).cuda()
    u = torch.tensor([1.0, float("nan"), float("inf"), 1.0]).to(KINDS[kind]).cuda()
    h = g.swiglu(bad, u)
    assert torch.isnan(h[0]) and torch.isnan(h[1]) and torch.isinf(h[2]) and torch.isfinite(h[3])


def test_large_factors_meet_a_small_slope():
    """dh u = 1e50 lies outside fp32, dh u s (1 + g (1 - s)) at these gates inside: below 1e37."""
    g = glowq()
    gate = torch.tensor([-75.0, -60.0, -50.0, -40.0, -35.0]).cuda()
    up, dh = torch.full_like(gate, 1e25), torch.full_like(gate, -1e25)
    (dg, bg), (du, bu) = R.swiglu_backward(dh, gate, up, "f32")
    a, c = g.swiglu_backward(dh, gate, up)
    R.within(a, dg, bg, "d_gate")
    R.within(c, du, bu, "d_up")


def test_gradients_against_differences():
    """Central differences in fp64 of the reference formula at step 1e-4: error below its third derivative's
    share, h^2 / 6 times at most 2 |dh u| (|g| + 3), plus the fp32 bound."""
    g = glowq()
    gate, up, dh = (values((500,), "f32", i) for i in range(3))
    a, c = g.swiglu_backward(dh, gate, up)
    G, U, D, s = gate.double(), up.double(), dh.double(), 1e-4
    f = lambda x, u: x / (1.0 + torch.exp(-x)) * u
    num = D * (f(G + s, U) - f(G - s, U)) / (2 * s)
    tol = (D * U).abs() * ((G.abs() + 3) * s * s + 2 * R.GATE * (1 + G.abs())) + 1e-30
    assert bool(((a.double() - num).abs() <= tol).all())
    num = D * (f(G, U + s) - f(G, U - s)) / (2 * s)
    assert bool(((c.double() - num).abs() <= (D * G).abs() * 2 * R.GATE + 1e-10).all())


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_in_place(kind):
    g = glowq()
    gate, up, dh = (values((33, 21), kind, i) for i in range(3))
    want, (dg, du) = g.swiglu(gate, up), g.swiglu_backward(dh, gate, up)
    for i in range(2):
        t = [gate.clone(), up.clone()]
        assert torch.equal(g.swiglu(*t, out=t[i]), want)
    t = [dh.clone(), gate.clone(), up.clone()]
    a, b = g.swiglu_backward(*t, out=(t[1], t[2]))
    assert torch.equal(a, dg) and torch.equal(b, du)


def test_empty_streams_and_graph():
    g = glowq()
    e = torch.empty(0, 5, dtype=torch.float16, device="cuda")
    assert g.swiglu(e, e).shape == (0, 5) and g.swiglu_backward(e, e, e)[0].shape == (0, 5)
    gate, up, dh = (values((300, 77), "f16", i) for i in range(3))
    want = [g.swiglu(gate, up), *g.swiglu_backward(dh, gate, up)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [g.swiglu(gate, up, stream=s), *g.swiglu_backward(dh, gate, up, stream=s)]
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [g.swiglu(gate, up), *g.swiglu_backward(dh, gate, up)]
    for k in range(3):
        gate.copy_(values((300, 77), "f16", 10 + k))
        want = [g.swiglu(gate, up), *g.swiglu_backward(dh, gate, up)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
