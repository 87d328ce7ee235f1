"""Block-scaled e4m3 weights past 2^31 and 2^32 bytes, dense and over 256 experts, and 256 experts of 7168 inputs: the rows and
experts at both ends and behind the places where 32 bits end, against the fp64 reference."""
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
    torch.cuda.empty_cache()


def codes(n, d, seed):
    """Random e4m3 bytes on the GPU, none NaN."""
    gen = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(0, 254, (n, d), dtype=torch.uint8, device="cuda", generator=gen)
    return q + (q > 126).to(torch.uint8)  # 0 .. 126 and 128 .. 254


@pytest.fixture(scope="module")
def big():
    g = glowq()
    n, d, r = 270001, 16384, 16
    q = codes(n, d, 1)
    gen = torch.Generator().manual_seed(2)
    s = 0.0001 + 0.0005 * torch.rand(-(-n // 128), d // 128, generator=gen)
    a, b = (0.3 * torch.randn(n, r, generator=gen)).half(), (torch.randn(r, d, generator=gen) / d ** 0.5).half()
    w = g.QWeight.from_fp8(q, s)
    # whole blocks of 128 rows: the first, around 2^31 and 2^32 bytes of codes, the last
    keep = [0, 1023, 1024, 2047, 2048, -(-n // 128) - 1]
    rows = torch.cat([torch.arange(128 * k, min(128 * k + 128, n)) for k in keep])
    yield n, d, r, w, a, b, rows, q[rows.cuda()].view(E4M3).cpu(), s[keep], a[rows]


@pytest.mark.parametrize("T", [1, 20, 48, 130])
def test_weights_past_32_bits(big, T):
    g = glowq()
    n, d, r, w, a, b, rows, q, s, a_kept = big
    x = (torch.randn(T, d, generator=torch.Generator().manual_seed(T)) * 0.5).half()
    log(f"fp8 {n} rows of {d}, T={T}")
    y = g.group_forward_fp8(x.cuda(), [w], b.cuda(), [a.cuda()], r)[0]
    ref, bound = F.product(x, q, s, b, a_kept, True)
    R.within(y[:, rows.cuda()], ref, bound, f"T={T}")


# (rows of a module, inputs, tokens, choices): single tokens, pieces, tiles; 4.6 GB, 2.1 GB and 0.7 GB of codes
@pytest.mark.parametrize("n,d,T,k", [(1100, 16384, 40, 8), (1100, 16384, 400, 8), (500, 16384, 5, 8), (400, 7168, 3, 8), (400, 7168, 60, 8),
                                     (400, 7168, 700, 8)])
@pytest.mark.parametrize("share", ["expert", "all"])
def test_experts_past_32_bits(n, d, T, k, share):
    g = glowq()
    E, r = 256, 16
    gen = torch.Generator().manual_seed(3)
    how = g.MOE_SHARE_EXPERT if share == "expert" else g.MOE_SHARE_ALL
    q = codes(E * n, d, 4)
    s = 0.0001 + 0.0005 * torch.rand(E, -(-n // 128), d // 128, generator=gen)
    a = (0.3 * torch.randn(E, n, r, generator=gen)).half().cuda()
    b = (torch.randn(*((E, r, d) if share == "expert" else (r, d)), generator=gen) / d ** 0.5).half()
    mod = g.MoeModule.stack([g.QWeight.from_fp8(q[e * n:(e + 1) * n], s[e]) for e in range(E)], list(a))
    x = (torch.randn(T, d, generator=gen) * 0.5).half()
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32)
    ids[0, : 4] = torch.tensor([0, 120, 239, 255], dtype=torch.int32)  # the choices that are checked have a row each
    ids[0, 4:] = torch.arange(1, k - 3)
    ws = g.init_workspace(torch.empty(g.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda"))
    offsets, token, _ = g.moe_sort(ids.cuda(), E, workspace=ws)
    log(f"fp8 256 experts, {n} rows of {d}, T={T} {share}")
    y = g.moe_forward_fp8(x.cuda(), E, [mod], b.cuda(), how, r, True, token, offsets, T * k)[0]
    off, tok = offsets.cpu(), token.cpu()
    for e in (0, 120, 239, 255):
        j = slice(int(off[e]), int(off[e + 1]))
        assert j.stop > j.start
        ref, bound = F.product(x[tok[j].long()], q[e * n:(e + 1) * n].view(E4M3).cpu(), s[e], b[e] if share == "expert" else b, a[e], True)
        R.within(y[j], ref, bound, f"expert {e}")
