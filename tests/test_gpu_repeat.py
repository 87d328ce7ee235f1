"""The block-scaled FP8 products, the router and the layer norm give the same bits again, whatever their workspace held before
and whatever ran between."""
import pytest
import torch

from gpu_util import glowq, log
from test_gpu_fp8 import Unit
from test_gpu_moe_fp8 import Layer
from test_gpu_moe_route import made as logits
from test_gpu_norm import made as rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


def same(call, ws, first=0):
    """call() gives the same bits for every filling of the workspace behind its first `first` bytes."""
    want = [t.clone() for t in call()]
    for fill in (0xFF, 0x00, 0x7B, 0xFF):
        if ws is not None:
            ws[first:] = fill
        big = torch.ones(1 << 22, device="cuda") * fill  # the caches hold something else
        got = call()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), hex(fill)
        del big


# every form of the group product
@pytest.mark.parametrize("T,d,rows_", [(1, 1024, [300, 20]), (30, 1024, [300]), (64, 1024, [1024, 512]), (48, 14336, [260]), (70, 14336, [300]),
                                       (300, 4096, [640]), (600, 512, [2600, 20]), (1300, 512, [2600, 2100]), (200, 640, [100])])
def test_fp8_group(T, d, rows_):
    g = glowq()
    u = Unit(T, d, rows_, 64, 1)
    ws = torch.empty(g.fp8_workspace_bytes(T, d, 64), dtype=torch.uint8, device="cuda")
    x, b, a = u.x.cuda(), u.b.cuda(), [t.cuda() for t in u.a]
    log(f"fp8 again T={T} d={d} {rows_}")
    same(lambda: g.group_forward_fp8(x, u.w, b, a, 64, workspace=ws), ws)


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [20, 33, 0, 7], [40, 30, 0, 20], [300, 0, 129, 200], [7] * 100])
@pytest.mark.parametrize("share", ["expert", "all"])
def test_fp8_experts(counts, share):
    g = glowq()
    how = g.MOE_SHARE_EXPERT if share == "expert" else g.MOE_SHARE_ALL
    T = max(counts)
    u = Layer(T, 384, [300, 70], counts, 24, how, 2)
    ws = g.init_workspace(torch.empty(g.moe_fp8_workspace_bytes(u.n, T, 384, 24, how), dtype=torch.uint8, device="cuda"))
    x, b, tok, off = u.x.cuda(), u.b.cuda(), u.token.cuda(), u.offsets.cuda()
    log(f"fp8 experts again {counts[:5]} {share}")
    same(lambda: g.moe_forward_fp8(x, u.E, u.mods, b, how, 24, True, tok, off, u.n, workspace=ws), ws, 8192)
    assert g.workspace_status(ws) == g.OK


@pytest.mark.parametrize("T,E,k,groups", [(1, 60, 4, 1), (700, 60, 4, 4), (500, 128, 8, 8), (400, 256, 8, 8), (300, 200, 20, 8)])
def test_route(T, E, k, groups):
    g = glowq()
    lo, bias = logits(T, E, "f32", 3, masked=True)
    lo, bias = lo.cuda(), bias.cuda()
    ws = g.init_workspace(torch.empty(8192, dtype=torch.uint8, device="cuda"))
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    log(f"route again T={T} E={E} k={k}")

    def call():
        ids, w = g.moe_route(lo, k, "sigmoid", bias, groups, max(1, groups // 2), 2, True, 2.5, ws)
        plain, pw = g.moe_route(lo, k, workspace=ws)
        return ids, w, plain, pw, g.moe_route_backward(dw, lo, ids, "sigmoid", True, 2.5, ws), g.moe_route_backward(dw, lo, plain, "softmax", False, 1.0, ws)
    same(call, None)
    assert g.workspace_status(ws) == g.OK


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 4096), (9000, 100), (8195, 250), (4100, 500), (2100, 1000), (1100, 2047), (700, 4095), (300, 8000), (270, 16384)])
def test_norm(T, d, kind):
    g = glowq()
    x, w, b, dy = rows(T, d, kind, 4)
    ws = torch.empty(g.layer_norm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    log(f"norm again {T}x{d} {kind}")

    def call():
        y = g.layer_norm(x, w, b)
        return y + g.layer_norm_backward(dy, x, y[1], y[2], w, ws)
    same(call, ws)
