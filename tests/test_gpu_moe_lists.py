"""Routed-row calls on lists that name too little or too much: which rows they write, and what they report."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import glowq, log
from test_gpu_moe_rows import KINDS, lists, randn, routing, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("bad", [30, -2, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("no_tokens", [False, True])
def test_combine_gradient_reports_tokens_out_of_range(bad, no_tokens):
    """row_token entries out of range are reported although no pair points at their row; the row given by
    the caller is left as it was."""
    g = glowq()
    T, k, d = (0, 2, 40) if no_tokens else (30, 2, 40)
    tok, pr, n = lists(30, 2, 5, 5)
    ws = workspace()
    if no_tokens:
        pr = pr[:0].contiguous()
        tok = torch.full_like(tok, -1)
    lone = 11
    p2 = torch.where(pr == lone, torch.full_like(pr, -1), pr)
    rows, dy, w = randn((n, d), "f32", 1), randn((T, d), "f32", 2), torch.rand(T, k).cuda()
    out = lambda: (torch.full((n, d), 3.0, device="cuda"), torch.empty(T, k, device="cuda"))
    g.moe_combine_backward(dy, rows, p2, tok, w, workspace=ws, out=out())
    assert g.workspace_status(ws) == g.OK
    tok = tok.clone()
    tok[lone] = bad
    log(f"token {bad} of row {lone}, T={T}")
    dr, _ = g.moe_combine_backward(dy, rows, p2, tok, w, workspace=ws, out=out())
    assert g.workspace_status(ws) == g.ERR_ROUTING
    assert bool((dr[lone] == 3.0).all())


def poisoned(shape, dtype):
    """Leaves NaN in the memory that the next allocation of this size gets."""
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("T,k,E,d,drop", [(1, 1, 1, 1, 0), (30, 2, 5, 40, 0.2), (300, 6, 9, 129, 0.3), (64, 64, 70, 24, 0.1),
                                          (2500, 4, 60, 2048, 0.1)])
def test_combine_gradient_of_fresh_memory_is_whole(T, k, E, d, drop, kind):
    """Without `out` every row is written: rows that no pair takes, rows of token -1 and rows of a token
    out of range get zeros, the others the gradient."""
    g = glowq()
    log(f"whole gradient T={T} k={k} E={E} d={d} {kind}")
    ids = routing(T, k, E, 7 + T, drop)
    off, tok, pr = g.moe_sort(ids.cuda(), E, workspace=workspace(T, k, E))
    n = T * k  # rows of token -1 behind the last expert's
    rows, dy = randn((n, d), kind, 1), randn((T, d), kind, 2)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(3)).cuda()
    gen = torch.Generator().manual_seed(4)
    p2, t2 = pr.cpu().clone(), tok.cpu().clone()
    p2[torch.rand(T, k, generator=gen) < 0.3] = -1
    bad = None
    if T > 1:
        bad = int(pr[pr >= 0][-1])
        t2[bad] = T + 5
    ws = workspace()
    poisoned((n, d), KINDS[kind])
    dr, dw = g.moe_combine_backward(dy, rows, p2.cuda(), t2.cuda(), w, workspace=ws)
    assert g.workspace_status(ws) == (g.OK if bad is None else g.ERR_ROUTING)
    use = p2.numpy().copy()
    if bad is not None:
        use[use == bad] = -1
    ref, bound, rw, bw, named = R.combine_backward(dy, rows, use, w.cpu().double().numpy(), n, kind)
    R.within(dr, ref, bound, "d_rows")
    R.within(dw, rw, bw, "d_weights")
    assert not dr[torch.from_numpy(~named).cuda()].any()


def test_combine_gradient_whole_in_place_and_captured():
    """The whole form on the rows' own memory through the C entry, and captured and replayed with lists
    that change between the replays."""
    g = glowq()
    T, k, E, d = 200, 3, 8, 72
    off, tok, pr = g.moe_sort(routing(T, k, E, 1, 0.1).cuda(), E, workspace=workspace(T, k, E))
    n = T * k
    rows, dy, w = randn((n, d), "f16", 1), randn((T, d), "f16", 2), torch.rand(T, k).cuda()
    ws = workspace()
    held_pr = pr.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            held = g.moe_combine_backward(dy, rows, held_pr, tok, w, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        gone = torch.rand(T, k, generator=torch.Generator().manual_seed(rep)) < 0.4
        held_pr.copy_(torch.where(gone.cuda(), torch.full_like(pr, -1), pr))
        for t in held:
            t.fill_(float("nan"))
        want = g.moe_combine_backward(dy, rows, held_pr, tok, w, workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        ref, bound, rw, bw, named = R.combine_backward(dy, rows, held_pr.cpu().numpy(), w.cpu().double().numpy(), n, "f16")
        R.within(want[0], ref, bound, "d_rows")
        for a, b in zip(held, want):
            assert torch.equal(a, b), rep
    r2, dw = rows.clone(), torch.empty(T, k, device="cuda")
    st = g.lib().glowq_moe_combine_backward_whole(dy.data_ptr(), r2.data_ptr(), n, held_pr.data_ptr(), tok.data_ptr(),
                                                  w.data_ptr(), T, k, d, g.DTYPE_F16, r2.data_ptr(), dw.data_ptr(),
                                                  ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == g.OK
    assert torch.equal(r2, want[0]) and torch.equal(dw, want[1])
    assert g.workspace_status(ws) == g.OK


def far_lists():
    """Calls without a workspace on lists with one entry out of range each, by name."""
    g = glowq()
    T, k, E, d = 30, 2, 5, 40
    tok, pr, n = lists(T, k, E, 5)
    ids = routing(T, k, E, 5).cuda()
    x, rows, dy, w = randn((T, d), "f16", 1), randn((n, d), "f16", 2), randn((T, d), "f16", 3), torch.rand(T, k).cuda()
    i2, t2, p2 = ids.clone(), tok.clone(), pr.clone()
    i2[3, 1], t2[4], p2[5, 0] = E, T, n
    return {"sort": lambda bad: g.moe_sort(i2 if bad else ids, E),
            "dispatch": lambda bad: g.moe_dispatch(x, t2 if bad else tok),
            "dispatch gradient": lambda bad: g.moe_dispatch_backward(rows, p2 if bad else pr),
            "combine": lambda bad: g.moe_combine(rows, p2 if bad else pr, w),
            "combine gradient": lambda bad: g.moe_combine_backward(dy, rows, p2 if bad else pr, tok, w)}


def status_of(f):
    """Status of a call.  The exception dies here: kept beside a graph (pytest.raises(...) as e) it would keep
    the frame, and so the graph, until the collector runs -- perhaps within another test's capture, where a
    graph must not be destroyed."""
    g = glowq()
    try:
        f()
    except g.GlowQError as err:
        return err.status
    return g.OK


NAMES = ["sort", "dispatch", "dispatch gradient", "combine", "combine gradient"]


@pytest.mark.parametrize("name", NAMES)
def test_without_workspace_list_errors_are_raised(name):
    """A call that makes its own workspace is the only one that can look at its error word."""
    g = glowq()
    f = far_lists()[name]
    log(f"no workspace: {name}")
    f(False)
    assert status_of(lambda: f(True)) == g.ERR_ROUTING
    f(False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert status_of(lambda: f(True)) == g.ERR_ROUTING
    torch.cuda.current_stream().wait_stream(s)


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls_need_a_workspace(name):
    """Under capture nobody could look at it: refused before anything is recorded, the capture goes on."""
    g = glowq()
    f = far_lists()[name]
    one = torch.ones(8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            status = status_of(lambda: f(False))
            two = one + one
    torch.cuda.current_stream().wait_stream(s)
    assert status == g.ERR_WORKSPACE
    graph.replay()
    torch.cuda.synchronize()
    assert bool((two == 2).all())
