"""Block-scaled e4m3 group forward (glowq_group_forward_fp8) against a plain fp64 reference: exact token codes and
scales in the workspace, every output within the bound of its roundings."""
import numpy as np
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


def blocks(n, d):
    return -(-n // 128), d // 128


class Unit:
    """Seeded e4m3 modules over d inputs with factors of rank r."""

    def __init__(self, T, d, rows, r, seed, extremes=False):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)
        self.T, self.d, self.rows, self.r = T, d, rows, r
        self.x = (rn(T, d) * (0.2 + rn(1, d).abs())).half()
        self.q = [(100 * rn(n, d)).clamp(-448, 448).to(E4M3) for n in rows]
        if extremes:
            for q in self.q:
                q[0] = 448.0
                q[-1] = -448.0
        self.s = [0.0001 + 0.0005 * torch.rand(*blocks(n, d), generator=gen) for n in rows]
        self.b = (rn(r, d) / d ** 0.5).half()
        self.a = [(rn(n, r) * 0.3).half() for n in rows]
        g = glowq()
        self.w = [g.QWeight.from_fp8(q, s) for q, s in zip(self.q, self.s)]

    def run(self, restore=True, x=None, **kw):
        g = glowq()
        x = self.x.cuda() if x is None else x
        on = restore and self.r > 0
        return g.group_forward_fp8(x, self.w, self.b.cuda() if on else None, [t.cuda() for t in self.a] if on else [],
                                   self.r, restore, **kw)

    def check(self, ys, restore, what):
        for i, (y, q, s, a) in enumerate(zip(ys, self.q, self.s, self.a)):
            ref, bound = F.product(self.x, q, s, self.b, a, restore and self.r > 0)
            R.within(y, ref, bound, f"{what} module {i}")


# one token to several token tiles of every kernel, ragged tokens and rows, blocks of 128 rows that end inside a tile, one
# to eight modules, one input group (d = 128) to many, ranks that fill no, part of and several correction steps
SHAPES = [(1, 128, [16], 0), (1, 256, [1], 8), (1, 4096, [520, 17, 130], 64), (2, 384, [40, 24], 8), (15, 1152, [100], 24),
          (16, 1024, [520, 17], 64), (17, 512, [96, 64, 40], 32), (31, 640, [33] * 8, 16), (33, 640, [100], 24),
          (48, 2176, [300], 128), (64, 1024, [1024, 512, 512], 64), (65, 256, [48, 32], 16), (130, 384, [300, 200], 40),
          (300, 512, [2048, 2048], 128), (8, 2048, [64], 256), (257, 896, [1030, 515], 64), (513, 128, [770], 256),
          (77, 14336, [128], 64), (40, 8192, [256], 8), (70, 2048, [130, 250], 64), (129, 4096, [640], 72), (1025, 640, [300], 0),
          (129, 1280, [4096, 20], 24), (300, 16384, [160], 8), (2100, 256, [4000], 24), (1400, 640, [2100, 2500, 1301], 0),
          (129, 4096, [4500], 72), (300, 16384, [700], 8), (130, 4224, [2000, 40], 24), (70, 14336, [1030], 64), (1100, 4096, [130], 0),
          (700, 512, [3100], 64), (1030, 384, [300, 200], 40), (1027, 128, [300], 256), (1026, 896, [1030, 515], 64),
          (1024, 128, [4100], 8), (4096, 4096, [20], 24), (4097, 256, [30], 8), (40, 1024, [9000], 24),
          (50, 640, [8300], 0), (48, 14336, [260], 72), (33, 12288, [40, 17], 8)]


@pytest.mark.parametrize("idx", range(len(SHAPES)), ids=[f"T{s[0]}_d{s[1]}_m{len(s[2])}_r{s[3]}" for s in SHAPES])
def test_forward(idx):
    T, d, rows, r = SHAPES[idx]
    u = Unit(T, d, rows, r, 100 + idx)
    for restore in ((True, False) if r else (False,)):
        log(f"fp8 T={T} d={d} rows={rows} r={r} restore={restore}")
        u.check(u.run(restore), restore, f"T={T} d={d} r={r}")


def test_codes_and_scales_in_the_workspace():
    g = glowq()
    for T, d in ((5, 128), (37, 640), (130, 4096)):
        u = Unit(T, d, [32], 0, 7)
        u.x[0] = 0
        u.x[1, :128] = 6e-8  # the smallest fp16
        u.x[2, :128] = torch.linspace(-65504, 65504, 128)
        u.x[3, :64] = 448.0
        u.x[3, 64:128] = torch.arange(64) * 0.5 + 0.25  # ties between codes
        ws = torch.full((g.fp8_workspace_bytes(T, d, 0),), 0xFF, dtype=torch.uint8, device="cuda")
        u.check(u.run(False, workspace=ws), False, "codes")
        torch.cuda.synchronize()
        ref, scale = F.quantise(u.x)
        assert np.array_equal(ws[: T * d].cpu().numpy().reshape(T, d), F.e4m3_bytes(ref))
        gp, at = -(-(d // 128) // 4) * 4, -(-T * d // 256) * 256
        got = ws[at: at + 4 * T * gp].view(torch.float32).cpu().numpy().reshape(T, gp)
        assert np.array_equal(got[:, : d // 128], scale) and (got[:, d // 128:] == 0).all()


def test_extremes_and_exact_sums():
    """Largest codes everywhere; one input a group, where every step is exact."""
    for T, rows in ((40, [64, 20]), (4100, [64, 20]), (260, [2100])):
        u = Unit(T, 2048, rows, 0, 3, extremes=True)
        u.check(u.run(False), False, f"extremes T={T}")
    for T in (1, 40, 150, 4100):
        u = Unit(T, 1024, [150], 0, 4)
        u.x[:] = 0
        u.x[:, ::128] = 2.0
        u.q = [torch.full_like(u.q[0].float(), 2.0).to(E4M3)]
        u.s = [torch.full_like(u.s[0], 0.25)]
        u.w = [glowq().QWeight.from_fp8(u.q[0], u.s[0])]
        y = u.run(False)[0]
        # scale 2 / 448 in fp32, code 448: eight groups of 448 * 2 * 0.25 * scale
        want = np.float32(0)
        for _ in range(8):
            want = np.float32(want + np.float32(np.float32(896) * np.float32(np.float32(2 / 448) * np.float32(0.25))))
        assert abs(float(y[0, 0]) - float(want)) <= 2.0 ** -11 * abs(float(want)) and (y == y[0, 0]).all()


@pytest.mark.parametrize("T", [1, 3, 30, 70, 200, 1700])
def test_nan_and_infinity_stay_in_their_token(T):
    u = Unit(T, 640, [300, 20], 16, 5)
    clean = u.run()
    for bad in (float("nan"), float("inf"), float("-inf")):
        x = u.x.clone()
        x[T // 2, 500] = bad
        ys = u.run(x=x.cuda())
        for y, c in zip(ys, clean):
            keep = torch.arange(T) != T // 2
            assert torch.isnan(y[T // 2]).all() and torch.equal(y[keep], c[keep])


def test_weights_bad_data_and_refusals():
    g = glowq()
    q = torch.zeros(130, 256).to(E4M3)
    s = torch.ones(2, 2)
    g.QWeight.from_fp8(q, s)
    g.QWeight.from_fp8(q.view(torch.uint8), s)
    for code in (0x7F, 0xFF):
        bad = q.view(torch.uint8).clone()
        bad[129, 255] = code
        with pytest.raises(g.GlowQError) as e:
            g.QWeight.from_fp8(bad, s)
        assert e.value.status == g.ERR_RANGE
    for v in (float("nan"), float("inf")):
        bad = s.clone()
        bad[1, 1] = v
        with pytest.raises(g.GlowQError) as e:
            g.QWeight.from_fp8(q, bad)
        assert e.value.status == g.ERR_RANGE
    for args in ((q, s[:1]), (q.float(), s), (q, s.double()), (q[:, :100], s), (q[0], s)):
        with pytest.raises(g.GlowQError):
            g.QWeight.from_fp8(*args)
    u = Unit(5, 256, [40], 8, 1)
    x, b, a = u.x.cuda(), u.b.cuda(), [t.cuda() for t in u.a]
    int8 = g.QWeight.from_int8(torch.zeros(40, 256, dtype=torch.int8), torch.ones(40))
    bad = [lambda: g.group_forward_fp8(x.float(), u.w, b, a, 8), lambda: g.group_forward_fp8(x, [int8], b, a, 8),
           lambda: g.group_forward_fp8(x, u.w + [int8], b, a + a, 8), lambda: g.group_forward_w8a8(x, u.w, b, a, 8),
           lambda: g.group_forward(x, u.w, b, a, 8), lambda: g.group_forward_fp8(x[:, :128], u.w, b, a, 8),
           lambda: g.group_forward_fp8(x, u.w, b[:4], a, 8), lambda: g.group_forward_fp8(x, u.w, None, a, 8),
           lambda: g.group_forward_fp8(x, u.w, b, [], 8), lambda: g.group_forward_fp8(x.cpu(), u.w, b, a, 8),
           lambda: g.group_forward_fp8(x, u.w, b, a, 8, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
           lambda: g.group_forward_fp8(x, u.w, b, a, 8, y=[torch.empty(5, 39, dtype=torch.float16, device="cuda")])]
    for f in bad:
        with pytest.raises(g.GlowQError):
            f()
    assert u.run(x=x[:0])[0].shape == (0, 40)


def test_large_workspace_streams_and_two_calls():
    """A workspace of the largest call for every smaller one; calls on two streams with a workspace each."""
    g = glowq()
    units = [Unit(T, 1024, [300, 260], 64, T) for T in (1100, 300, 70, 20, 1)]
    ws = torch.full((g.fp8_workspace_bytes(1100, 1024, 64),), 0xFF, dtype=torch.uint8, device="cuda")
    for u in units:
        u.check(u.run(workspace=ws), True, f"T={u.T}")
    want = [u.run() for u in units[:2]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        got = [u.run(stream=s) for u, s in zip(units, streams)]
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(p, q))


@pytest.mark.parametrize("T,d", [(1, 1024), (24, 1024), (70, 1024), (300, 1024), (70, 14336), (300, 4096), (1100, 1024), (48, 14336)])
def test_captured_and_replayed(T, d):
    g = glowq()
    u = Unit(T, d, [300, 760], 64, T)
    ws = torch.empty(g.fp8_workspace_bytes(T, d, 64), dtype=torch.uint8, device="cuda")
    x, b, a = u.x.cuda(), u.b.cuda(), [t.cuda() for t in u.a]
    call = lambda: g.group_forward_fp8(x, u.w, b, a, 64, workspace=ws)
    eager = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = call()
    for seed in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ys, eager))
        x.copy_(torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).half())
        eager = call()
