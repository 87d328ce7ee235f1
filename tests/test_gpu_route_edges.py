"""The router where rows, biases and scores end: rows without a choice in the gradient, standings of groups that cancel,
rows of the type's lowest value, renormalised sigmoids too small for a number."""
import math

import numpy as np
import pytest
import torch

import layer_ref as R
import router_ref as Q
from gpu_util import glowq, log
from test_gpu_moe_route import KINDS, check, made, ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("E,k", [(60, 4), (128, 8), (250, 16), (200, 40)])
def test_gradient_of_rows_without_a_choice_is_zero(E, k, kind):
    """Rows that the router refused (NaN, +inf), rows of -inf alone and rows whose choices are all of experts that are out:
    no choice is live, so that the row is zeros whatever its logits and its weights' gradients are."""
    g = glowq()
    lo, _ = made(12, E, kind, 5)
    clean = lo.clone()
    lo[1, 7], lo[3, E - 1], lo[4], lo[6, 0] = math.nan, math.inf, -math.inf, math.nan
    lo[8, :k] = -math.inf
    none = [1, 3, 4, 6, 8]
    rest = [t for t in range(12) if t not in none]
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            log(f"route gradient without a choice {E} {k} {kind} {score} renorm={renorm}")
            w_ = ws()
            ids, _ = g.moe_route(lo.cuda(), k, score, renorm=renorm, workspace=w_)
            assert g.workspace_status(w_) == g.ERR_ROUTING
            assert (ids[[1, 3, 4, 6]] == -1).all()
            ids[8] = torch.arange(k, dtype=torch.int32)  # experts of logit -inf
            dw = torch.randn(12, k, generator=torch.Generator().manual_seed(3))
            dw[4] = math.nan
            got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids, score, renorm, 2.5, w_)
            assert g.workspace_status(w_) == g.OK
            assert (got[none] == 0).all(), (score, renorm, got[none].isnan().any(1).tolist())
            ref, bound = Q.route_backward(dw[rest], clean[rest], ids[rest], score, renorm, 2.5, kind)
            R.within(got[rest], ref, bound, f"{score} renorm={renorm}")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1.0, 30.0, 100.0, 1000.0, 1e6])
def test_standings_that_cancel(size, score):
    """Groups by their two best, which have a bias of B and one of -B (B of its own for every group): the sum is about that of two
    scores, its error in fp32 that of B, and the groups' scores are as far apart as such an error.  The other experts are out."""
    gen = torch.Generator().manual_seed(int(size))
    for E, G, keep in ((16, 4, 1), (64, 8, 3), (256, 16, 7)):
        n, T = E // G, 400
        lo = torch.full((T, E), -math.inf)
        bias = torch.zeros(E)
        for grp in range(G):
            B = size * float(torch.rand((), generator=gen))
            a, b = (grp * n + torch.randperm(n, generator=gen)[:2]).tolist()
            lo[:, a], lo[:, b] = (1e-6 * size * torch.randn(T, generator=gen) for _ in range(2))
            bias[a], bias[b] = B, -B
        log(f"cancelling standings {score} B={size} E={E}")
        check(lo, 2 * keep, score, bias, G, keep, 2, what=f"cancelling {E}")


def test_standings_past_the_largest_number():
    """Biases of the type's lowest value: a group that they hold down still stands above a group without experts, and its two
    best add up to more than fp32 holds."""
    low = -3.4028234663852886e38
    lo = torch.randn(20, 16, generator=torch.Generator().manual_seed(1))
    lo[:, :4] = -math.inf
    lo[:10, 4:6] = -math.inf
    bias = torch.zeros(16)
    bias[8:] = low
    for score in ("softmax", "sigmoid"):
        for keep in (1, 2, 3):
            for best in (1, 2):
                check(lo, 8, score, bias, 4, keep, best, what=f"{score} {keep} {best}")
        check(lo, 8, score, -bias, 4, 2, 2, what=f"{score} largest")


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("E,k", [(60, 4), (128, 8), (256, 8), (100, 20)])
def test_rows_of_the_lowest_value(E, k, kind):
    """Logits masked with the type's lowest value instead of -inf: experts of a row of it alone share it evenly, and beside others
    they have no weight."""
    g = glowq()
    low = torch.finfo(KINDS[kind]).min
    lo, b = made(9, E, kind, 6)
    lo[0] = low
    lo[1], lo[1, : k + 2] = -math.inf, low
    lo[2], lo[2, 5] = low, 1.0
    lo[3, ::2] = low
    lo[4], lo[4, 3] = low, low / 2
    lo[5], lo[5, 3] = -math.inf, low
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for bias, G, keep, best in ((None, 1, 1, 1), (b, 1, 1, 1), (b, 4, 2, 2), (None, 4, 2, 2)):
                log(f"lowest {E} {k} {kind} {score} renorm={renorm} bias={bias is not None} groups={G}")
                ids, w = check(lo, k, score, bias, G, keep, best, renorm, 1.0, f"{score} renorm={renorm}")
                if renorm:
                    assert (w.sum(1) - 1).abs().max() < 1e-5
                if score == "softmax":
                    live = float((lo[0] == low).sum())
                    assert (w[0] - (1 / k if renorm else 1 / live)).abs().max() < 1e-6
                dw = torch.randn(9, k, generator=torch.Generator().manual_seed(3))
                got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids, score, renorm, 1.0, ws())
                assert torch.isfinite(got).all()
                ref, bound = Q.route_backward(dw, lo, ids, score, renorm, 1.0, kind)
                R.within(got, ref, bound, f"gradient {score} renorm={renorm}")


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_renormalised_sigmoids_below_the_smallest_number(kind):
    """Chosen logits whose sigmoids are subnormal or zero in fp32 beside ones that are not: the weights are ratios, with the
    bits of any other."""
    g = glowq()
    rows = [[-75.0, -90.0, -95.0, -100.0], [-75.0, -100.0, -76.0, -75.5], [-20.0, -100.0, -105.0, -90.0], [-17.0, -101.5, -16.5, -17.5],
            [-79.9, -103.0, -104.0, -110.0], [-80.1, -103.0, -104.0, -110.0], [-1.0, -85.0, -88.0, -0.5], [-5.0, -92.0, -88.5, -90.0],
            [0.0, -20.0, -80.0, -86.0], [30.0, -20.0, -50.0, 16.0], [-87.0, -103.9, -104.1, -130.0], [-0.0, -1e-3, 1e-3, -12.0]]
    lo = torch.full((len(rows), 20), -math.inf)
    lo[:, 3:7] = torch.tensor(rows)
    lo = lo.to(KINDS[kind])
    for bias in (None, torch.linspace(-1, 1, 20)):
        for scale in (1.0, 2.5):
            check(lo, 4, "sigmoid", bias, scale=scale, what="small sigmoids")
            check(lo, 3, "sigmoid", bias, scale=scale, what="small sigmoids, three")
    for k in (2, 3, 4):
        ids, _ = g.moe_route(lo.cuda(), k, "sigmoid")
        dw = torch.randn(len(rows), k, generator=torch.Generator().manual_seed(3))
        got = g.moe_route_backward(dw.cuda(), lo.cuda(), ids, "sigmoid", True, 2.5, ws())
        ref, bound = Q.route_backward(dw, lo, ids, "sigmoid", True, 2.5, kind)
        R.within(got, ref, bound, f"gradient {k}")
