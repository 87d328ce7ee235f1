"""Block-scaled e4m3 products on inputs that are far apart inside one group: the matrix step adds eight products at the
largest one's exponent and drops what lies 13 bits below it, so that a large input leaves its seven neighbours few bits.  Every
form stays within the bound that says so, and the distance from the exact results is printed."""
import numpy as np
import pytest
import torch

import fp8_ref as F
import layer_ref as R
from gpu_util import glowq, log
from test_gpu_fp8 import E4M3, Unit
from test_gpu_moe_fp8 import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


def apart(x, how, seed):
    """x [T][d] with large inputs 300 times the others: "one" in each group, "eights" one in every eight, "cancel" the same value
    in every eight (its weights cancel)."""
    gen = torch.Generator().manual_seed(seed)
    T, d = x.shape
    x = torch.randn(T, d, generator=gen) * 0.05
    at = torch.arange(0, d, 128 if how == "one" else 8) + 3
    x[:, at] = 15.0 if how == "cancel" else 15.0 * torch.randn(T, at.numel(), generator=gen)
    return x.half(), at


def weights(q, at, how):
    q = q.float()
    if how == "cancel":
        q[:, at] = torch.where(torch.arange(at.numel()) % 2 == 0, 448.0, -448.0)
    return q.to(E4M3)


def distance(y, ref):
    return float(np.linalg.norm(R.f64(y) - ref) / np.linalg.norm(ref))


# every form of the group product: pieces of 16 and 32 tokens, tiles of 64, 128 x 128 with K ranges, 128 x 256
SHAPES = [(1, 1024, [260]), (30, 512, [300, 40]), (48, 14336, [260]), (70, 14336, [300]), (300, 4096, [640]), (1300, 512, [2600, 2100])]


@pytest.mark.parametrize("how", ["one", "eights", "cancel"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[0]}_d{s[1]}")
def test_group_products_of_inputs_far_apart(shape, how):
    g = glowq()
    T, d, rows = shape
    u = Unit(T, d, rows, 16, 11)
    u.x, at = apart(u.x, how, T)
    u.q = [weights(q, at, how) for q in u.q]
    u.w = [g.QWeight.from_fp8(q, s) for q, s in zip(u.q, u.s)]
    ys = u.run(False)
    off = [distance(y, F.product(u.x, q, s, u.b, a, False)[0]) for y, q, s, a in zip(ys, u.q, u.s, u.a)]
    log(f"fp8 far apart {how} T={T} d={d}: {max(off):.2e} of the norm")
    u.check(ys, False, how)
    u.check(u.run(True), True, how)


@pytest.mark.parametrize("how", ["one", "eights", "cancel"])
@pytest.mark.parametrize("counts", [[1, 0, 2], [20, 33, 0], [140, 0, 90]], ids=lambda c: "rows" + "_".join(map(str, c)))
def test_experts_products_of_inputs_far_apart(counts, how):
    g = glowq()
    u = Layer(50, 640, [300, 70], counts, 16, g.MOE_SHARE_EXPERT, 3)
    u.x, at = apart(u.x, how, 5)
    u.q = [[weights(q, at, how) for q in qs] for qs in u.q]
    u.mods = [g.MoeModule.stack([g.QWeight.from_fp8(q, s) for q, s in zip(qs, ss)], [t.cuda() for t in aa])
              for qs, ss, aa in zip(u.q, u.s, u.a)]
    log(f"fp8 experts far apart {how} {counts}")
    u.check(u.run(False), False, how)
    u.check(u.run(True), True, how)
