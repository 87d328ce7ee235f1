"""Routing lists, the rows' way into expert order and back, and their gradients against plain fp64
references: lists equal value for value, rows within the bound of their roundings."""
import numpy as np
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


def workspace(T=1, k=1, E=1):
    g = glowq()
    return g.init_workspace(torch.empty(g.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda"))


def routing(T, k, E, seed, drop=0.0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.topk(torch.rand(T, E, generator=gen), k, 1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    if drop:
        ids[torch.rand(T, k, generator=gen) < drop] = -1
    return ids


def check_sort(ids, E, ws=None):
    g = glowq()
    T, k = ids.shape
    got = g.moe_sort(ids.cuda(), E, workspace=workspace(T, k, E) if ws is None else ws)
    for name, a, b in zip(("offsets", "row_token", "pair_row"), got, R.sort(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b), name
    return got


# one pair, one wavefront, one workgroup (8192 pairs) and beyond, experts filling part of and whole
# bucket words, more choices than experts named twice
@pytest.mark.parametrize("T,k,E,drop", [
    (0, 4, 60, 0), (1, 1, 1, 0), (1, 4, 60, 0), (3, 2, 2, 0.5), (16, 4, 60, 0), (63, 1, 3, 0.2), (257, 4, 64, 0),
    (1024, 8, 256, 0.1), (2048, 4, 60, 0), (8191, 1, 255, 0), (2049, 4, 63, 0.3), (5000, 6, 128, 0), (40001, 2, 256, 0.05)])
def test_sort_lists(T, k, E, drop):
    log(f"sort T={T} k={k} E={E} drop={drop}")
    check_sort(routing(T, k, E, T + E, drop), E)


@pytest.mark.parametrize("n", [500, 20000])
def test_sort_one_expert_all_dropped_and_repeats(n):
    check_sort(torch.full((n, 1), 5, dtype=torch.int32), 7)
    off, tok, pr = check_sort(torch.full((n, 1), -1, dtype=torch.int32), 7)
    assert int(off[-1]) == 0 and bool((tok == -1).all()) and bool((pr == -1).all())
    check_sort(torch.randint(0, 3, (n, 4), dtype=torch.int32, generator=torch.Generator().manual_seed(n)), 3)


@pytest.mark.parametrize("n", [100, 12000])
def test_sort_reports_ids_out_of_range(n):
    g = glowq()
    ws = workspace(n, 1, 9)
    ids = routing(n, 1, 9, 3)
    check_sort(ids, 9, ws)
    assert g.workspace_status(ws) == g.OK
    for bad in (9, -2, 2 ** 31 - 1, -2 ** 31):
        ids[n // 2] = bad
        check_sort(ids, 9, ws)  # such pairs take no row
        assert g.workspace_status(ws) == g.ERR_ROUTING
        assert g.workspace_status(ws) == g.OK


def lists(T, k, E, seed, drop=0.0):
    g = glowq()
    ids = routing(T, k, E, seed, drop)
    off, tok, pr = g.moe_sort(ids.cuda(), E, workspace=workspace(T, k, E))
    n = int(off[-1])
    return tok[:n].contiguous(), pr, n


def randn(shape, kind, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(KINDS[kind]).cuda()


# d: single values, rows that are and are not multiples of 16 bytes, one and several passes of a workgroup
SIZES = [(1, 1, 1, 1, 0), (1, 4, 60, 2048, 0), (5, 2, 4, 17, 0.3), (64, 4, 8, 64, 0), (33, 8, 16, 1001, 0.2),
         (200, 3, 60, 4096, 0.1), (700, 4, 60, 130, 0), (7, 5, 9, 9000, 0), (300, 1, 3, 8, 0.5), (4, 64, 100, 24, 0.1)]


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("T,k,E,d,drop", SIZES)
def test_rows_and_gradients(T, k, E, d, drop, kind):
    g = glowq()
    log(f"rows T={T} k={k} E={E} d={d} {kind} drop={drop}")
    tok, pr, n = lists(T, k, E, 50 + T + d, drop)
    ws = workspace()
    x, rows, add, dy = (randn(s, kind, i) for i, s in enumerate(((T, d), (n, d), (T, d), (T, d))))
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(9)).cuda()
    prn, wn = pr.cpu().numpy(), w.cpu().double().numpy()
    got = g.moe_dispatch(x, tok, workspace=ws)
    assert torch.equal(got, x[tok.long()])
    for weights, base in ((w, add), (w, None), (None, None)):
        y, bound = R.combine(rows, prn, None if weights is None else wn, base, kind)
        R.within(g.moe_combine(rows, pr, weights, add=base, workspace=ws), y, bound, "combine")
    y, bound = R.combine(rows, prn, None, None, kind)
    R.within(g.moe_dispatch_backward(rows, pr, workspace=ws), y, bound, "dispatch gradient")
    for weights in (w, None):
        dr, drb, dw, dwb, named = R.combine_backward(dy, rows, prn, None if weights is None else wn, n, kind)
        assert named.all()
        a, b = g.moe_combine_backward(dy, rows, pr, tok, weights, workspace=ws)
        R.within(a, dr, drb, "d_rows")
        R.within(b, dw, dwb, "d_weights")
    assert g.workspace_status(ws) == g.OK


@pytest.mark.parametrize("kind,d,T,k", [("f16", 4096, 2500, 2), ("f16", 4095, 900, 6), ("f32", 2052, 900, 6),
                                        ("f32", 2051, 2500, 2)])
def test_rows_that_outgrow_the_caches(kind, d, T, k):
    """More than 32 MB of rows (read past the caches): every row of sampled tokens."""
    g = glowq()
    tok, pr, n = lists(T, k, 12, 33, 0.05)
    assert n * d * (2 if kind == "f16" else 4) > 32 << 20
    ws = workspace()
    rows, dy = randn((n, d), kind, 1), randn((T, d), kind, 2)
    w = torch.rand(T, k).cuda()
    some = torch.arange(0, T, 43)
    y = g.moe_combine(rows, pr, w, add=dy, workspace=ws)
    dr, dw = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws)
    dx = g.moe_dispatch_backward(rows, pr, workspace=ws)
    prs, ws_ = pr.cpu()[some].numpy(), w.cpu()[some].double().numpy()
    R.within(y[some], *R.combine(rows, prs, ws_, dy[some], kind), "combine")
    R.within(dx[some], *R.combine(rows, prs, None, None, kind), "dispatch gradient")
    assert torch.equal(g.moe_dispatch(dy, tok, workspace=ws), dy[tok.long()])
    ref, bound, rw, bw, named = R.combine_backward(dy[some], rows, prs, ws_, n, kind)
    R.within(dr[torch.from_numpy(named).cuda()], ref[named], bound[named], "d_rows")
    R.within(dw[some], rw, bw, "d_weights")
    assert g.workspace_status(ws) == g.OK


def test_gradients_against_differences():
    """<dy, combine(rows + h v) - combine(rows - h v)> / 2h against <d_rows, v>, and the same for weights:
    the operator is linear in each, so in fp32 only rounding is left (values of order 1, h = 1)."""
    g = glowq()
    T, k, E, d = 40, 3, 8, 96
    tok, pr, n = lists(T, k, E, 3, 0.1)
    ws = workspace()
    rows, dy, v = (randn(s, "f32", i) for i, s in enumerate(((n, d), (T, d), (n, d))))
    w, u = torch.rand(T, k).cuda(), torch.rand(T, k).cuda()
    dr, dw = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws)
    f = lambda r, q: float((g.moe_combine(r, pr, q, workspace=ws).double() * dy.double()).sum())
    # T d products, each of fp32 values with up to 2 (k + 1) roundings of sums below 2 k max|w| max|row|
    scale = float(dy.double().abs().sum()) * k * float(rows.abs().max() + v.abs().max())
    tol = scale * 2 * (k + 2) * R.U32
    assert abs((f(rows + v, w) - f(rows - v, w)) / 2 - float((dr.double() * v.double()).sum())) <= tol
    assert abs((f(rows, w + u) - f(rows, w - u)) / 2 - float((dw.double() * u.double()).sum())) <= 2 * tol


def test_tail_rows_and_unnamed_rows():
    """Lists of T top_k rows where pairs were dropped: rows behind the last expert's have token -1 -- zero
    rows, zero gradients.  A row no pair takes keeps what its gradient held; a token without rows gets
    `add`, or zeros."""
    g = glowq()
    ws = workspace()
    ids = routing(50, 4, 6, 21, 0.4)
    ids[7] = -1
    off, tok, pr = g.moe_sort(ids.cuda(), 6, workspace=ws)
    n, live = 200, int(off[-1])
    x, rows, dy = (randn(s, "f16", i) for i, s in enumerate(((50, 72), (n, 72), (50, 72))))
    w = torch.rand(50, 4).cuda()
    got = g.moe_dispatch(x, tok, workspace=ws)
    assert torch.equal(got[:live], x[tok[:live].long()]) and not got[live:].any()
    assert torch.equal(g.moe_combine(rows, pr, w, add=dy, workspace=ws)[7], dy[7])
    assert not g.moe_combine(rows, pr, w, workspace=ws)[7].any()
    out = (torch.full((n, 72), 3.0, dtype=torch.float16, device="cuda"), torch.empty(50, 4, device="cuda"))
    dr, dw = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws, out=out)
    assert not dr[live:].any() and not dw[7].any()
    lone = int(pr[pr >= 0][0])
    pr2 = torch.where(pr == lone, torch.full_like(pr, -1), pr)
    out[0].fill_(3.0)
    dr, _ = g.moe_combine_backward(dy, rows, pr2, tok, w, workspace=ws, out=out)
    assert bool((dr[lone] == 3.0).all())
    assert g.workspace_status(ws) == g.OK


def test_no_tokens_but_rows():
    """Padded row lists of a batch without tokens: every row zero, forward and backward."""
    g = glowq()
    ws = workspace()
    tok = torch.full((300,), -1, dtype=torch.int32, device="cuda")
    none, rows = torch.empty(0, 24, device="cuda"), torch.full((300, 24), 5.0, device="cuda")
    got = g.moe_dispatch(none, tok, workspace=ws, out=rows.clone())
    assert got.shape == (300, 24) and not got.any()
    pr = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    dr, dw = g.moe_combine_backward(none, rows, pr, tok, None, workspace=ws, out=(rows.clone(), torch.empty(0, 3, device="cuda")))
    assert not dr.any() and dw.shape == (0, 3)
    assert g.workspace_status(ws) == g.OK


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_in_place(kind):
    """y in add, d_rows in rows."""
    g = glowq()
    tok, pr, n = lists(40, 6, 9, 3)
    ws = workspace()
    rows, dy, w = randn((n, 50), kind, 1), randn((40, 50), kind, 2), torch.rand(40, 6).cuda()
    want = g.moe_combine(rows, pr, w, add=dy, workspace=ws)
    y = dy.clone()
    assert torch.equal(g.moe_combine(rows, pr, w, add=y, workspace=ws, out=y), want)
    dr, dw = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws)
    r = rows.clone()
    a, b = g.moe_combine_backward(dy, r, pr, tok, w, workspace=ws, out=(r, torch.empty(40, 6, device="cuda")))
    assert torch.equal(a, dr) and torch.equal(b, dw) and g.workspace_status(ws) == g.OK


def test_bad_list_entries_are_skipped_and_reported():
    g = glowq()
    T, k, E, d = 30, 2, 5, 40
    tok, pr, n = lists(T, k, E, 5)
    ws = workspace()
    x, rows, dy = (randn(s, "f32", i) for i, s in enumerate(((T, d), (n, d), (T, d))))
    w = torch.rand(T, k).cuda()
    for bad in (T, -2, 2 ** 31 - 1):
        t2 = tok.clone()
        t2[4] = bad
        got = g.moe_dispatch(x, t2, workspace=ws)
        want = x[tok.long()]
        want[4] = 0
        assert torch.equal(got, want) and g.workspace_status(ws) == g.ERR_ROUTING
    clean = g.moe_combine(rows, pr, w, workspace=ws)
    dr0, dw0 = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws)
    assert g.workspace_status(ws) == g.OK
    for bad in (n, -2, 2 ** 31 - 1, -2 ** 31):
        p2 = pr.clone()
        p2[3, 1] = bad
        y = g.moe_combine(rows, p2, w, workspace=ws)
        assert g.workspace_status(ws) == g.ERR_ROUTING
        ref, bound = R.combine(rows, np.where(np.arange(T * k).reshape(T, k) == 3 * k + 1, -1, pr.cpu().numpy()),
                               w.cpu().double().numpy(), None, "f32")
        R.within(y, ref, bound, "skipped")
        assert torch.equal(y[:3], clean[:3]) and torch.equal(y[4:], clean[4:])
        out = (torch.full((n, d), 7.0, device="cuda"), torch.empty(T, k, device="cuda"))
        dr, dw = g.moe_combine_backward(dy, rows, p2, tok, w, workspace=ws, out=out)
        assert g.workspace_status(ws) == g.ERR_ROUTING
        assert float(dw[3, 1]) == 0.0 and bool((dr[int(pr[3, 1])] == 7.0).all())
    # the same row twice: by another token (row_token names one), and by two choices of one token
    for t, j, src in ((9, 0, pr[2, 1]), (9, 1, pr[9, 0])):
        p2 = pr.clone()
        p2[t, j] = src
        out = (torch.full((n, d), 7.0, device="cuda"), torch.empty(T, k, device="cuda"))
        dr, dw = g.moe_combine_backward(dy, rows, p2, tok, w, workspace=ws, out=out)
        assert g.workspace_status(ws) == g.ERR_ROUTING
        assert torch.equal(dr[int(src)], dr0[int(src)]) and float(dw[t, j]) == 0.0
        assert bool((dr[int(pr[t, j])] == 7.0).all())


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_non_finite_values_stay_in_their_token(kind):
    g = glowq()
    tok, pr, n = lists(20, 2, 4, 6)
    ws = workspace()
    rows = randn((n, 64), kind, 1)
    w = torch.rand(20, 2).cuda()
    clean = g.moe_combine(rows, pr, w, workspace=ws)
    r2 = rows.clone()
    r2[int(pr[5, 0]), 3] = float("inf")
    r2[int(pr[8, 1]), 9] = float("nan")
    y = g.moe_combine(r2, pr, w, workspace=ws)
    assert torch.isinf(y[5, 3]) and torch.isnan(y[8, 9])
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[5, 3] = keep[8, 9] = False
    assert torch.equal(y[keep], clean[keep])


def test_graph_replays_and_streams():
    """Sort, dispatch, combine and the gradients in one captured graph, replayed with new ids and eager
    calls between; and on another stream than the current one."""
    g = glowq()
    T, k, E, d = 3000, 4, 60, 128
    ws, ws2 = workspace(T, k, E), workspace(T, k, E)
    ids = routing(T, k, E, 0).cuda()
    x, dy, w = randn((T, d), "f16", 1), randn((T, d), "f16", 2), torch.rand(T, k).cuda()

    def layer(ws, stream=None):
        off, tok, pr = g.moe_sort(ids, E, workspace=ws, stream=stream)
        rows = g.moe_dispatch(x, tok, workspace=ws, stream=stream)
        y = g.moe_combine(rows, pr, w, add=x, workspace=ws, stream=stream)
        dr, dw = g.moe_combine_backward(dy, rows, pr, tok, w, workspace=ws, stream=stream)
        return [off, tok, pr, rows, y, dr, dw, g.moe_dispatch_backward(dr, pr, workspace=ws, stream=stream)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held = layer(ws)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        ids.copy_(routing(T, k, E, 100 + rep))
        want = layer(ws2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), rep
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = layer(ws2, other)
    other.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_without_workspace_and_large_rows():
    """No workspace given; offsets past 2^31 bytes (70000 rows of 16384 fp32 values), sampled."""
    g = glowq()
    T, k, E, d = 35000, 2, 16, 16384
    ids = torch.topk(torch.rand(T, E, device="cuda"), k, 1).indices.to(torch.int32)
    off, tok, pr = g.moe_sort(ids, E)
    x = torch.randn(T, d, device="cuda")
    rows = g.moe_dispatch(x, tok)
    for i in (0, 33000, 40000, 69999):
        assert torch.equal(rows[i], x[int(tok[i])])
    w = torch.rand(T, k, device="cuda")
    y = g.moe_combine(rows, pr, w)
    for t in (0, 17000, T - 1):
        want = x[t].double() * w[t].double().sum()
        assert bool(((y[t].double() - want).abs() <= 4 * (k + 1) * R.U32 * want.abs() + 1e-30).all())
    dr, dw = g.moe_combine_backward(x, rows, pr, tok, w)
    for t in (0, 20000, T - 1):
        for j in range(k):
            p = w[t, j] * x[t]
            assert torch.equal(dr[int(pr[t, j])], p)
            n2 = float((x[t].double() ** 2).sum())
            assert abs(float(dw[t, j]) - n2) <= d * R.U32 * n2
