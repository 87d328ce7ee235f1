"""Layer norm and its gradients on more rows than the workgroups take at once (every form's loop over its rows, the next row
requested ahead), past the 32 MB from which they bypass the caches, on rows of odd length, and in place there."""
import pytest
import torch

import layer_ref as R
import router_ref as Q
from gpu_util import glowq, log
from test_gpu_norm import made

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    glowq()
    yield
    torch.cuda.synchronize()


# the forward takes 2048 workgroups' rows at once, the gradients 256 (of 16, 16, 4, 4, 1 ... and 64, 32, 16, 8, 4, 2, 1, 1 rows a
# workgroup by columns): two turns and more, the last one ragged
LOOPS = [(33001, 100), (33001, 130), (8195, 511), (8195, 700), (2051, 1100), (2051, 2500), (2050, 4097)]
# past 32 MB in either type, and two turns and more
PAST = [(132107, 127), (65801, 255), (32835, 511), (16403, 1023), (8199, 2047), (4100, 4095), (2051, 8191), (2051, 16383)]


def both(x, w, b, dy, kind, what):
    g = glowq()
    y, mean, rstd = g.layer_norm(x, w, b, 1e-5)
    for got, (ref, bound), name in zip((y, mean, rstd), Q.norm(x, w, b, 1e-5, kind), ("y", "mean", "rstd")):
        R.within(got, ref, bound, f"{what} {name}")
    back = g.layer_norm_backward(dy, x, mean, rstd, w)
    for got, (ref, bound), name in zip(back, Q.norm_backward(dy, x, mean, rstd, w, kind), ("dx", "dw", "db")):
        R.within(got, ref, bound, f"{what} {name}")
    return (y, mean, rstd), back


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("shape", LOOPS, ids=lambda s: "x".join(map(str, s)))
def test_more_rows_than_workgroups(shape, kind):
    log(f"norm {shape} {kind}")
    x, w, b, dy = made(*shape, kind, 3)
    both(x, w, b, dy, kind, "loop")


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("shape", PAST, ids=lambda s: "x".join(map(str, s)))
def test_past_the_caches(shape, kind):
    T, d = shape
    if kind == "f32" and d < 8191:
        T = -(-T // 2)
    log(f"norm {(T, d)} {kind}")
    x, w, b, dy = made(T, d, kind, 4)
    both(x, w, b, dy, kind, "past the caches")


@pytest.mark.parametrize("shape", [(33001, 100), (8195, 511), (2051, 1100), (8199, 2047), (4100, 4095), (2051, 16383)],
                         ids=lambda s: "x".join(map(str, s)))
def test_in_place(shape):
    """The forward onto x, the gradient onto x and onto dy: the bits of the calls into other memory, twice."""
    g = glowq()
    x, w, b, dy = made(*shape, "f16", 5)
    log(f"norm in place {shape}")
    y, mean, rstd = g.layer_norm(x, w, b)
    dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(2):
        xx = x.clone()
        got = g.layer_norm(xx, w, b, out=(xx, torch.empty_like(mean), torch.empty_like(rstd)))
        assert all(torch.equal(p, q) for p, q in zip(got, (y, mean, rstd)))
        for into in ("x", "dy"):
            xx, gg = x.clone(), dy.clone()
            got = g.layer_norm_backward(gg, xx, mean, rstd, w, None, (xx if into == "x" else gg, torch.empty_like(dw), torch.empty_like(db)))
            assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db))), into
