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
