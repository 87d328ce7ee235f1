"""8-bit integer group forward (glowq_group_forward_w8a8) against a plain fp64 reference: exact token
codes and scales in the workspace, every output within the bound of its roundings."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import glowq, log
from oracle import glowq_ref as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


class Unit:
    """Seeded int8 modules over d inputs with factors of rank r."""

    def __init__(self, T, d, rows, r, seed, extremes=False):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)
        self.T, self.d, self.rows, self.r = T, d, rows, r
        self.x = (rn(T, d) * (0.2 + rn(1, d).abs())).half()
        self.codes = [torch.randint(-128, 128, (n, d), generator=gen, dtype=torch.int32).to(torch.int8) for n in rows]
        if extremes:
            for q in self.codes:
                q[0] = -128
                q[-1] = 127
        self.scales = [0.001 + 0.002 * torch.rand(n, generator=gen) for n in rows]
        self.b = (rn(r, d) / d ** 0.5).half()
        self.a = [(rn(n, r) * 0.3).half() for n in rows]
        g = glowq()
        self.w = [g.QWeight.from_int8(q, s) for q, s in zip(self.codes, self.scales)]

    def run(self, restore=True, x=None, **kw):
        g = glowq()
        x = self.x.cuda() if x is None else x
        on = restore and self.r > 0
        return g.group_forward_w8a8(x, self.w, self.b.cuda() if on else None, [t.cuda() for t in self.a] if on else [],
                                    self.r, restore, **kw)

    def check(self, ys, restore, what):
        ref, bound = R.w8a8(self.x, self.codes, self.scales, self.b, self.a, restore and self.r > 0)
        for i, (y, yr, bd) in enumerate(zip(ys, ref, bound)):
            R.within(y, yr, bd, f"{what} module {i}")


# one token to several token tiles of every kernel, ragged tokens and rows, one to eight modules,
# one input group (d = 128) to many, ranks that fill no, part of and several correction steps
SHAPES = [(1, 128, [16], 0), (1, 256, [1], 8), (1, 4096, [520, 17, 130], 64), (2, 384, [40, 24], 8), (15, 1152, [100], 24),
          (16, 1024, [520, 17], 64), (17, 512, [96, 64, 40], 32), (31, 640, [33] * 8, 16), (33, 640, [100], 24),
          (48, 2176, [300], 128), (64, 1024, [1024, 512, 512], 64), (65, 256, [48, 32], 16), (130, 384, [300, 200], 40),
          (300, 512, [2048, 2048], 128), (8, 2048, [64], 256), (257, 896, [1030, 515], 64), (513, 128, [770], 256),
          (700, 1280, [2050], 8), (96, 14336, [272], 64), (5, 16384, [48], 64), (33, 512, [16400, 1], 24),
          (64, 384, [8200, 8190], 64), (41, 128, [17000], 0)]


@pytest.mark.parametrize("T,d,rows,r", SHAPES)
def test_w8a8_matches_reference(T, d, rows, r):
    u = Unit(T, d, rows, r, 1000 + T + d)
    g = glowq()
    for restore in (True, False):
        n = g.w8a8_workspace_bytes(T, d, r if restore else 0)
        ws = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")  # the contents need no initialisation
        log(f"w8a8 T={T} d={d} rows={rows} r={r} restore={restore}")
        ys = u.run(restore, workspace=ws)
        torch.cuda.synchronize()
        codes, scale = G.quantize_x_int8(u.x)
        raw = ws.cpu().numpy()
        assert np.array_equal(raw[: T * d].view(np.int8).reshape(T, d), codes)
        o = (T * d + 255) // 256 * 256
        assert np.array_equal(raw[o: o + 4 * T].view(np.uint32), scale.astype(np.float32).reshape(-1).view(np.uint32))
        u.check(ys, restore, f"restore={restore}")


# input groups shared out unevenly: over K ranges (103 in 26 26 26 25, 17 in 9 8, 25 in 9 9 7) and over the teams
# of wavefronts inside a workgroup (26 in 7 7 7 5, 17 in 9 8), projections in several ranges, r up to 256
@pytest.mark.parametrize("T,d,rows,r", [(40, 13184, [130, 5], 24), (64, 16384, [272], 256), (33, 16384, [1024, 8], 0),
                                        (128, 2176, [17000], 40), (66, 2048, [16500, 3], 200), (300, 2176, [5000], 64),
                                        (200, 3200, [600, 30], 200), (500, 16384, [140], 8), (60, 4224, [9000], 72)])
def test_w8a8_uneven_splits(T, d, rows, r):
    u = Unit(T, d, rows, r, 3000 + T + d)
    log(f"w8a8 uneven T={T} d={d} rows={rows} r={r}")
    u.check(u.run(r > 0), r > 0, "uneven")


# the projection's blocks of 16 and 32 tokens: both sides of the rule that chooses them, ragged tokens and ranks
@pytest.mark.parametrize("T,d,rows,r", [(128, 16384, [48], 256), (129, 8192, [48], 256), (145, 16384, [33], 200),
                                        (200, 15744, [40], 64), (199, 15744, [40], 64), (300, 10496, [16, 7], 8),
                                        (299, 10496, [16, 7], 8), (640, 1280, [17], 256), (1537, 2048, [130], 72)])
def test_w8a8_projection_blocks(T, d, rows, r):
    u = Unit(T, d, rows, r, 5000 + T + d)
    log(f"w8a8 projection blocks T={T} d={d} rows={rows} r={r}")
    u.check(u.run(), True, "blocks")


@pytest.mark.parametrize("T,d,rows,r", [(2048, 512, [4096, 1000], 64), (2043, 384, [4096, 4090], 24),
                                        (1500, 256, [9000, 3001], 0), (1100, 640, [16400], 128),
                                        (70001, 128, [520], 8), (66000, 256, [20], 64)])
def test_w8a8_large_grid(T, d, rows, r):
    """Grids of the large tiles, every token block: tokens sampled from each 64 against the reference."""
    u = Unit(T, d, rows, r, 7 + T)
    some = torch.cat([torch.arange(0, T, 37), torch.tensor([T - 1])])
    ys = u.run(r > 0)
    sub = Unit.__new__(Unit)
    sub.__dict__.update(u.__dict__)
    sub.x = u.x[some]
    sub.check([y[some.cuda()] for y in ys], r > 0, f"large T={T}")


@pytest.mark.parametrize("T", [2, 40, 70])
def test_w8a8_weights_past_four_gigabytes(T):
    """270000 x 16384 codes: byte offsets of the last rows' blocks need more than 32 bits."""
    g = glowq()
    n, d, r = 270000, 16384, 8
    gen = torch.Generator("cuda").manual_seed(T)
    codes = torch.randint(-128, 128, (n, d), generator=gen, dtype=torch.int8, device="cuda")
    scales = 0.001 + 0.002 * torch.rand(n, generator=gen, device="cuda")
    x = torch.randn(T, d, generator=gen, device="cuda").half()
    b = (torch.randn(r, d, generator=gen, device="cuda") / d ** 0.5).half()
    a = (0.3 * torch.randn(n, r, generator=gen, device="cuda")).half()
    w = g.QWeight.from_int8(codes, scales)
    log(f"w8a8 past 4 GB T={T}")
    y, = g.group_forward_w8a8(x, [w], b, [a], r)
    some = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 262159, 269990, n - 1], device="cuda")
    ref, bound = R.w8a8(x.cpu(), [codes[some].cpu()], [scales[some].cpu()], b.cpu(), [a[some].cpu()], True)
    R.within(y[:, some], ref[0], bound[0], "far rows")


def test_w8a8_largest_sums_are_exact():
    """d = 16384 with every weight code -128 or 127 and equal activations: the largest int32 sums."""
    T, d = 18, 16384
    u = Unit(T, d, [32], 0, 8, extremes=True)
    u.codes[0][: 16] = -128
    u.codes[0][16:] = 127
    u.x = torch.ones(T, d).half()
    u.x[3] = -1.0
    g = glowq()
    u.w = [g.QWeight.from_int8(u.codes[0], u.scales[0])]
    u.check(u.run(False), False, "extremes")


@pytest.mark.parametrize("T", [3, 20, 70, 300])
def test_w8a8_zero_and_non_finite_tokens(T):
    """A zero token: zeros plus its (zero) correction.  A token with an infinity or a NaN: NaN in its
    own rows, no other row changed."""
    u = Unit(T, 512, [96, 33], 16, 9)
    u.x[1] = 0
    for restore in (True, False):
        clean = u.run(restore)
        u.check(clean, restore, f"zero token restore={restore}")
        x = u.x.clone()
        x[0, 5] = float("inf")
        x[2, 511] = float("nan")
        ys = u.run(restore, x=x.cuda())
        for y, c in zip(ys, clean):
            assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all()
            assert torch.equal(y[1], c[1]) and torch.equal(y[3:], c[3:])


@pytest.mark.parametrize("T", [2, 70])
def test_w8a8_overflowing_outputs_are_infinite(T):
    u = Unit(T, 256, [40], 0, 10)
    big = [s * 3e6 for s in u.scales]
    g = glowq()
    u.w = [g.QWeight.from_int8(u.codes[0], big[0])]
    y = u.run(False)[0].cpu()
    ref, _ = R.w8a8(u.x, u.codes, big, None, [], False)
    far = np.abs(ref[0]) > 66000.0
    assert far.any() and torch.isinf(y[torch.from_numpy(far)]).all()
    assert np.array_equal(np.sign(ref[0][far]), np.sign(y.double().numpy()[far]))


def test_w8a8_empty_and_repeatable():
    u = Unit(40, 384, [72, 16], 32, 11)
    assert [tuple(y.shape) for y in u.run(True, x=u.x.cuda()[:0])] == [(0, 72), (0, 16)]
    a, b = u.run(True), u.run(True)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("T", [1, 16, 33, 100, 600])
def test_w8a8_tokens_do_not_depend_on_the_batch(T):
    """The integer sums are exact whatever the tile: without the correction a token's row is the same
    bit for bit in every batch size."""
    u = Unit(600, 1024, [400], 0, 12)
    full = u.run(False)[0]
    part = u.run(False, x=u.x.cuda()[:T].contiguous())[0]
    assert torch.equal(part, full[:T])


def test_w8a8_repack_on_another_stream():
    """Transposed codes: their dense copy and the repack both on the given stream."""
    g = glowq()
    u = Unit(3, 4096, [2048], 0, 21)
    s = torch.cuda.Stream()
    codes, scales = u.codes[0].t().contiguous().cuda().t(), u.scales[0].cuda()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        w = g.QWeight.from_int8(codes, scales, stream=s)
        assert torch.equal(w.q, u.w[0].q) and torch.equal(w.sz[: 4 * 2048], u.w[0].sz[: 4 * 2048])


def test_w8a8_repack_rejects_non_finite_scales():
    g = glowq()
    for v in (float("inf"), float("nan")):
        s = torch.ones(20)
        s[13] = v
        with pytest.raises(g.GlowQError) as e:
            g.QWeight.from_int8(torch.zeros(20, 128, dtype=torch.int8), s)
        assert e.value.status == g.ERR_RANGE


@pytest.mark.parametrize("T", [1, 40, 400])
def test_w8a8_graph_replays_and_streams(T):
    """A captured call replayed with new inputs and eager calls between, and a call on another stream
    than the current one, equal the eager call bit for bit."""
    u = Unit(T, 1024, [272, 48], 64, 13)
    g = glowq()
    x = u.x.cuda()
    b, a = u.b.cuda(), [t.cuda() for t in u.a]
    ws = torch.empty(g.w8a8_workspace_bytes(T, 1024, 64), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(T, n, dtype=torch.float16, device="cuda") for n in u.rows]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.group_forward_w8a8(x, u.w, b, a, 64, workspace=ws, y=ys)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.group_forward_w8a8(x, u.w, b, a, 64, workspace=ws, y=ys)
    torch.cuda.current_stream().wait_stream(s)
    for k in range(4):
        x.copy_(torch.roll(u.x.cuda(), k, 1))
        want = g.group_forward_w8a8(x, u.w, b, a, 64)
        for y in ys:
            y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for y, v in zip(ys, want):
            assert torch.equal(y, v), k
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = g.group_forward_w8a8(x, u.w, b, a, 64, stream=other)
    other.synchronize()
    for y, v in zip(got, want):
        assert torch.equal(y, v)
