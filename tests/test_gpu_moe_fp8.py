"""The experts' product on block-scaled e4m3 weights (glowq_moe_forward_fp8) against a plain fp64 reference, expert by
expert."""
import pytest
import torch

import fp8_ref as F
import layer_ref as R
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


class Layer:
    """Seeded experts; counts: rows of each expert (tokens at random, repeated where rows outnumber them)."""

    def __init__(self, T, d, rows, counts, r, share, seed, listed=True):
        g = glowq()
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)
        self.T, self.d, self.rows, self.r, self.share, self.E = T, d, rows, r, share, len(counts)
        self.counts, self.n = counts, sum(counts)
        self.x = (rn(T, d) * (0.2 + rn(1, d).abs())).half()
        self.token = torch.randint(0, T, (self.n,), generator=gen).to(torch.int32) if listed else None
        self.offsets = torch.tensor([sum(counts[:e]) for e in range(self.E + 1)], dtype=torch.int32)
        self.q = [[(100 * rn(n, d)).clamp(-448, 448).to(E4M3) for _ in counts] for n in rows]
        self.s = [[0.0001 + 0.0005 * torch.rand(-(-n // 128), d // 128, generator=gen) for _ in counts] for n in rows]
        self.a = [[(rn(n, r) * 0.3).half() for _ in counts] for n in rows]
        self.b = (rn(self.E, r, d) / d ** 0.5).half() if share == g.MOE_SHARE_EXPERT else (rn(r, d) / d ** 0.5).half()
        self.mods = [g.MoeModule.stack([g.QWeight.from_fp8(q, s) for q, s in zip(qs, ss)], [t.cuda() for t in aa])
                     for qs, ss, aa in zip(self.q, self.s, self.a)]

    def run(self, restore=True, token="own", offsets=None, x=None, **kw):
        g = glowq()
        token = self.token if isinstance(token, str) else token
        return g.moe_forward_fp8((self.x if x is None else x).cuda(), self.E, self.mods, self.b.cuda() if self.r else None, self.share,
                                 self.r, restore, None if token is None else token.cuda(),
                                 (self.offsets if offsets is None else offsets).cuda(), self.n, **kw)

    def check(self, ys, restore, what, token="own"):
        g = glowq()
        token = self.token if isinstance(token, str) else token
        for i, y in enumerate(ys):
            for e in range(self.E):
                j = slice(int(self.offsets[e]), int(self.offsets[e + 1]))
                if j.start == j.stop:
                    continue
                x = self.x[j] if token is None else self.x[token[j].long()]
                b = self.b[e] if self.share == g.MOE_SHARE_EXPERT else self.b
                ref, bound = F.product(x, self.q[i][e], self.s[i][e], b, self.a[i][e], restore and self.r > 0)
                R.within(y[j], ref, bound, f"{what} module {i} expert {e}")


# (tokens, inputs, rows of the modules, rows listed for each expert, rank): single tokens, empty experts, experts of one
# row, ragged blocks of every form, one expert, many
SHAPES = [(1, 256, [40, 24], [0, 1, 0, 1], 8), (1, 2048, [130], [1, 1, 1, 1], 64), (3, 128, [16], [3], 0), (7, 640, [100, 30], [0, 0, 5, 2, 7], 24),
          (20, 384, [300], [16, 17, 0, 1], 40), (64, 1024, [130, 130], [33, 0, 64, 31], 64), (50, 512, [257], [70, 65, 3], 16),
          (200, 256, [520, 40], [200, 129, 0, 128, 1, 127], 128), (300, 1152, [140], [300, 260], 256), (90, 128, [33, 17, 50, 20], [90, 44], 8),
          (513, 256, [128], [513, 0, 0, 100], 72), (10, 16384, [20], [6, 4], 8)]


@pytest.mark.parametrize("share", ["expert", "all"])
@pytest.mark.parametrize("idx", range(len(SHAPES)), ids=[f"T{s[0]}_d{s[1]}_e{len(s[3])}_r{s[4]}" for s in SHAPES])
def test_forward(idx, share):
    g = glowq()
    T, d, rows, counts, r = SHAPES[idx]
    u = Layer(T, d, rows, counts, r, g.MOE_SHARE_EXPERT if share == "expert" else g.MOE_SHARE_ALL, 10 + idx)
    for restore in ((True, False) if r else (False,)):
        log(f"fp8 experts T={T} d={d} rows={rows} counts={counts} r={r} {share} restore={restore}")
        u.check(u.run(restore), restore, share)


def test_many_experts_and_rows_in_order():
    """256 experts, and the form without a token list (row j reads token j)."""
    g = glowq()
    counts = [(7 * e) % 5 for e in range(256)]
    u = Layer(40, 128, [20], counts, 8, g.MOE_SHARE_EXPERT, 1)
    u.check(u.run(), True, "256 experts")
    for counts in ([3, 0, 40], [150, 131]):
        for share in (g.MOE_SHARE_EXPERT, g.MOE_SHARE_ALL):
            u = Layer(sum(counts), 256, [140], counts, 16, share, 2, listed=False)
            u.check(u.run(), True, "in order")


@pytest.mark.parametrize("share", ["expert", "all"])
@pytest.mark.parametrize("E,T,d,rows,r", [(128, 20, 256, [300], 40), (43, 60, 384, [600, 24], 72), (128, 90, 128, [257, 40], 0), (64, 400, 128, [260, 300], 256)])
def test_large_tiles_of_few_rows(E, T, d, rows, r, share):
    """Many experts of about 11, 19, 11 and 20 rows each: tiles that are mostly empty; few tokens and their shared projection."""
    g = glowq()
    counts = [(7 * e) % (23 if E == 128 else 39) for e in range(E)]
    u = Layer(T, d, rows, counts, r, g.MOE_SHARE_EXPERT if share == "expert" else g.MOE_SHARE_ALL, 5)
    log(f"fp8 experts E={E} T={T} d={d} rows={rows} listed={u.n} r={r} {share}")
    u.check(u.run(), True, share)


def test_many_rows_of_few_experts():
    g = glowq()
    u = Layer(700, 128, [40], [2100, 0, 4133, 5], 72, g.MOE_SHARE_EXPERT, 6)
    u.check(u.run(), True, "many rows")


@pytest.mark.parametrize("counts", [[3, 2, 0], [140, 0, 150]])
def test_lists_out_of_range_are_clamped_and_reported(counts):
    g = glowq()
    for share in (g.MOE_SHARE_EXPERT, g.MOE_SHARE_ALL):
        u = Layer(20, 256, [40], counts, 8, share, 3)
        ws = g.init_workspace(torch.empty(g.moe_fp8_workspace_bytes(u.n, 20, 256, 8, share), dtype=torch.uint8, device="cuda"))
        good = u.run(workspace=ws)[0]
        assert g.workspace_status(ws) == g.OK
        for at, v in ((0, -1), (u.n - 1, 20), (1, 1 << 30), (1, -(1 << 31))):
            token = u.token.clone()
            token[at] = v
            y = u.run(token=token, workspace=ws)[0]
            assert g.workspace_status(ws) == g.ERR_ROUTING
            keep = torch.arange(u.n) != at
            assert torch.equal(y[keep], good[keep])
        for off in ([0, 1, u.n + 5, u.n], [-3, 1, 1, u.n], [0, 4, 2, u.n], [0, 1, 2, u.n - 1], [1 << 30] * 4, [0, -5, 1 << 30, -1]):
            u.run(offsets=torch.tensor(off, dtype=torch.int32), workspace=ws)
            assert g.workspace_status(ws) == g.ERR_ROUTING
        with pytest.raises(g.GlowQError):
            u.run(offsets=torch.tensor([0, 1, 2, u.n - 1], dtype=torch.int32))
        # rows that no expert covers stay as they were
        y = [torch.full((u.n, 40), 7.0, dtype=torch.float16, device="cuda")]
        off = u.offsets.clone()
        off[3] = off[2] = u.n - 1
        off[1] = min(int(off[1]), u.n - 1)
        u.run(offsets=off, workspace=ws, y=y)
        assert (y[0][u.n - 1] == 7.0).all() and g.workspace_status(ws) == g.ERR_ROUTING


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [40, 30, 0, 20], [300, 0, 129, 200]])
def test_captured_replayed_and_on_streams(counts):
    g = glowq()
    T = max(counts)
    u = Layer(T, 512, [150, 70], counts, 16, g.MOE_SHARE_EXPERT, 3)
    ws = g.init_workspace(torch.empty(g.moe_fp8_workspace_bytes(u.n, T, 512, 16, u.share), dtype=torch.uint8, device="cuda"))
    x, b, tok, off = u.x.cuda(), u.b.cuda(), u.token.cuda(), u.offsets.cuda()
    call = lambda **kw: g.moe_forward_fp8(x, u.E, u.mods, b, u.share, 16, True, tok, off, u.n, workspace=ws, **kw)
    eager = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = call(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = call()
    for seed in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ys, eager))
        x.copy_(torch.randn(T, 512, generator=torch.Generator().manual_seed(seed)).half())
        eager = call()
    assert g.workspace_status(ws) == g.OK


def test_nan_stays_in_its_rows():
    g = glowq()
    for counts in ([2, 3], [130, 140]):
        u = Layer(30, 256, [40], counts, 8, g.MOE_SHARE_EXPERT, 3)
        good = u.run()[0]
        x = u.x.clone()
        x[4, 200] = float("inf")
        y = u.run(x=x)[0]
        hit = u.token == 4
        assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], good[~hit])


def test_refusals():
    g = glowq()
    u = Layer(6, 256, [40], [3, 4], 8, g.MOE_SHARE_EXPERT, 3)
    x, b, tok, off = u.x.cuda(), u.b.cuda(), u.token.cuda(), u.offsets.cuda()
    ws = g.init_workspace(torch.empty(g.moe_fp8_workspace_bytes(7, 6, 256, 8, u.share), dtype=torch.uint8, device="cuda"))
    ok = lambda **k: g.moe_forward_fp8(**{**dict(x=x, n_exp=2, modules=u.mods, b=b, share=u.share, r=8, restore=True, row_token=tok, offsets=off,
                                                n_rows=7, workspace=ws), **k})
    ok()
    int4 = g.MoeModule(u.mods[0].q, u.mods[0].sz, u.mods[0].a, 40, 256)
    bad = [dict(x=x.float()), dict(x=x[:, :128]), dict(n_exp=3), dict(modules=[int4]), dict(modules=u.mods * 5), dict(modules=[]), dict(b=b[0]),
           dict(b=None), dict(r=16), dict(row_token=tok.long()), dict(offsets=off.long()), dict(offsets=off[:2]), dict(row_token=tok[:6]),
           dict(n_rows=-1), dict(workspace=ws[:8192]), dict(share=2), dict(row_token=None), dict(y=[torch.empty(6, 40, device="cuda").half()]),
           dict(y=[]), dict(x=x.cpu())]
    for k in bad:
        with pytest.raises(g.GlowQError):
            ok(**k)
            print("accepted", list(k))
    with pytest.raises(g.GlowQError):
        g.moe_forward(x, 2, u.mods, b, u.share, 8, True, tok, off, 7)
    with pytest.raises(g.GlowQError):
        g.MoeModule.stack([g.QWeight.from_fp8(u.q[0][0], u.s[0][0]), g.QWeight.from_int8(torch.zeros(40, 256, dtype=torch.int8), torch.ones(40))], None)
    assert ok(n_rows=0, row_token=tok[:0], offsets=off * 0)[0].shape == (0, 40)
