"""The block-scaled e4m3 group forward, the experts' product on such weights and their repacking without a GPU: sizes, and
every refusal before any HIP call."""
import ctypes

import pytest

from rank_error_compensation_amd import glowq as g

FAKE = 0x10000   # aligned fake device address: never dereferenced, validation fails first
HDR = 8192


def r256(n):
    return (n + 255) // 256 * 256


def test_weight_sizes():
    L = g.lib()
    assert L.glowq_fp8_q_bytes(4096, 4096) == 4096 * 4096
    assert L.glowq_fp8_q_bytes(17, 256) == 2 * 16 * 256   # whole strips of 16 rows
    assert L.glowq_fp8_sz_bytes(128, 4096) == 32 * 4
    assert L.glowq_fp8_sz_bytes(129, 256) == 64           # 2 x 2 scales, padded
    for n, k in ((0, 128), (16, 100), (16, 0), (16, 16384 + 128), ((1 << 24) + 1, 128), (-1, 128)):
        assert L.glowq_fp8_q_bytes(n, k) == 0 and L.glowq_fp8_sz_bytes(n, k) == 0


def test_workspace_bytes():
    f = g.lib().glowq_fp8_workspace_bytes
    assert f(3, 256, 0) >= r256(3 * 256) + r256(3 * 4 * 4)   # codes, four scales a token
    assert f(3, 256, 64) > f(3, 256, 0)
    for T, d, r in ((0, 256, 0), (-1, 256, 0), (3, 100, 0), (3, 16384 + 128, 0), (3, 256, -8), (3, 256, 264),
                    ((1 << 20) + 1, 128, 0)):
        assert f(T, d, r) == 0
    # a workspace for the largest call serves every smaller one
    Ts = [1, 2, 16, 31, 32, 33, 63, 64, 65, 100, 511, 512, 513, 1023, 1024, 1025, 4096, 4097, 8191, 8193, 65536]
    for d in (128, 2048, 4096, 11008, 16384):
        for r in (0, 8, 64, 72, 256):
            n = [f(T, d, r) for T in Ts]
            assert n == sorted(n), (d, r)
            assert r == 256 or all(f(T, d, r) <= f(T, d, r + 8) for T in Ts)
            assert d == 16384 or all(f(T, d, r) <= f(T, d + 128, r) for T in Ts)


def test_experts_workspace_bytes():
    f = g.lib().glowq_moe_fp8_workspace_bytes
    assert f(0, 0, 128, 0, 0) >= HDR
    assert f(16, 4, 256, 0, 0) >= HDR + r256(4 * 256) + r256(4 * 4 * 4)
    for n, T, d, r, share in ((-1, 4, 256, 0, 0), ((1 << 23) + 1, 4, 256, 0, 0), (16, -1, 256, 0, 0), (16, (1 << 20) + 1, 128, 0, 0),
                              (16, 4, 100, 0, 0), (16, 4, 0, 0, 0), (16, 4, 16512, 0, 0), (16, 4, 256, -8, 0), (16, 4, 256, 264, 0),
                              (16, 4, 256, 8, 2), (16, 4, 256, 8, -1)):
        assert f(n, T, d, r, share) == 0
    Ns = [1, 4, 31, 32, 33, 100, 2048, 8191, 8192, 8193, 16380, 100000]
    for share in (g.MOE_SHARE_EXPERT, g.MOE_SHARE_ALL):
        for r in (0, 8, 64, 72, 256):
            sizes = [f(n, 40, 2048, r, share) for n in Ns]
            assert sizes == sorted(sizes)
            sizes = [f(4000, T, 2048, r, share) for T in Ns]
            assert sizes == sorted(sizes)


def fp8(fmt=5, n_out=32, k_in=256, q=FAKE, sz=FAKE, reserved=0):
    return g.QWeightC(q, sz, n_out, k_in, fmt, reserved)


def forward(x=FAKE, T=4, d=256, w=None, m=None, b=FAKE, a=FAKE, r=8, restore=1, ws=FAKE, n=1 << 30, y=FAKE):
    w = [fp8()] if w is None else w
    m = len(w) if m is None else m
    wc = (g.QWeightC * max(1, len(w)))(*w)
    ac = (ctypes.c_void_p * max(1, len(w)))(*([a] * max(1, len(w))))
    yc = (ctypes.c_void_p * max(1, len(w)))(*([y] * max(1, len(w))))
    return g.lib().glowq_group_forward_fp8(x, T, d, m, wc, b, ac, r, restore, ws, n, yc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), g.ERR_INVALID_ARG), (dict(y=None), g.ERR_INVALID_ARG), (dict(a=None), g.ERR_INVALID_ARG),
    (dict(b=None), g.ERR_INVALID_ARG), (dict(w=[fp8(q=None)]), g.ERR_INVALID_ARG),
    (dict(w=[fp8(sz=None)]), g.ERR_INVALID_ARG), (dict(w=[fp8(fmt=6)]), g.ERR_INVALID_ARG),
    (dict(w=[fp8(fmt=-1)]), g.ERR_INVALID_ARG), (dict(w=[fp8(reserved=1)]), g.ERR_INVALID_ARG),
    (dict(w=[fp8(fmt=0)]), g.ERR_UNSUPPORTED), (dict(w=[fp8(fmt=1)]), g.ERR_UNSUPPORTED), (dict(w=[fp8(fmt=4)]), g.ERR_UNSUPPORTED),
    (dict(w=[fp8(), fp8(fmt=4)]), g.ERR_UNSUPPORTED), (dict(w=[fp8()] * 8, m=9), g.ERR_UNSUPPORTED),
    (dict(m=0), g.ERR_SHAPE), (dict(T=-1), g.ERR_SHAPE), (dict(d=100), g.ERR_SHAPE), (dict(d=0), g.ERR_SHAPE),
    (dict(w=[fp8(k_in=128)]), g.ERR_SHAPE), (dict(w=[fp8(n_out=0)]), g.ERR_SHAPE), (dict(r=-8), g.ERR_SHAPE),
    (dict(r=12), g.ERR_UNSUPPORTED), (dict(r=264), g.ERR_UNSUPPORTED),
    (dict(d=16512, w=[fp8(k_in=16512)]), g.ERR_UNSUPPORTED),
    (dict(T=1 << 20, d=2048, w=[fp8(k_in=2048)]), g.ERR_UNSUPPORTED),
    (dict(x=FAKE + 8), g.ERR_ALIGN), (dict(y=FAKE + 8), g.ERR_ALIGN), (dict(b=FAKE + 8), g.ERR_ALIGN),
    (dict(a=FAKE + 8), g.ERR_ALIGN), (dict(w=[fp8(q=FAKE + 4)]), g.ERR_ALIGN), (dict(ws=FAKE + 16), g.ERR_ALIGN),
    (dict(ws=None), g.ERR_WORKSPACE), (dict(n=64), g.ERR_WORKSPACE), (dict(restore=0, n=64), g.ERR_WORKSPACE),
    (dict(T=0), g.OK),
])
def test_group_refusals(kw, status):
    assert forward(**kw) == status


def test_every_other_entry_point_refuses_these_weights():
    L, big = g.lib(), 1 << 30
    wc = (g.QWeightC * 1)(fp8())
    p = (ctypes.c_void_p * 1)(FAKE)
    unit = (g.UnitC * 1)(g.UnitC(1, 1, FAKE, 4, 256, wc, FAKE, p, 8, 1, p))
    for r in (0, 8):
        assert L.glowq_solo_forward(FAKE, 4, 256, wc, FAKE, FAKE, r, 1, FAKE, big, FAKE, None) == g.ERR_INVALID_ARG
        assert L.glowq_group_forward_static(FAKE, 4, 256, 1, wc, FAKE, p, r, 1, p, None) == g.ERR_INVALID_ARG
        for f in (L.glowq_group_forward, L.glowq_group_forward_w4a8, L.glowq_group_forward_mx8, L.glowq_group_forward_w8a8):
            assert f(FAKE, 4, 256, 1, wc, FAKE, p, r, 1, FAKE, big, p, None) == g.ERR_INVALID_ARG
        assert L.glowq_layerwise_forward(FAKE, 4, 256, 1, wc, p, p, r, 1, FAKE, big, p, None) == g.ERR_INVALID_ARG
    assert L.glowq_path_forward(unit, 1, FAKE, big, None) == g.ERR_INVALID_ARG
    assert L.glowq_dequant(ctypes.byref(wc[0]), FAKE, 0, None) == g.ERR_INVALID_ARG
    assert L.glowq_ner_sums(FAKE, wc, FAKE, big, FAKE, None) in (g.ERR_INVALID_ARG, g.ERR_UNSUPPORTED)


def module(q=FAKE, sz=FAKE, a=FAKE, y=FAKE, n_out=64, k_in=256):
    return g.MoeModuleC(q, sz, a, y, n_out, k_in)


def experts(x=FAKE, T=8, d=256, n_exp=4, m=None, mods=None, b=FAKE, share=0, r=16, restore=1, tok=FAKE, off=FAKE, n_rows=16, ws=FAKE,
            n=1 << 24):
    mods = [module(), module()] if mods is None else mods
    c = (g.MoeModuleC * max(1, len(mods)))(*mods)
    return g.lib().glowq_moe_forward_fp8(x, T, d, n_exp, len(mods) if m is None else m, c, b, share, r, restore, tok, off, n_rows, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_exp=0), g.ERR_UNSUPPORTED), (dict(n_exp=257), g.ERR_UNSUPPORTED), (dict(m=5), g.ERR_UNSUPPORTED), (dict(m=0), g.ERR_UNSUPPORTED),
    (dict(share=2), g.ERR_INVALID_ARG), (dict(d=100), g.ERR_SHAPE), (dict(T=-1), g.ERR_SHAPE), (dict(T=0), g.ERR_SHAPE),
    (dict(n_rows=-1), g.ERR_SHAPE), (dict(n_rows=(1 << 23) + 1), g.ERR_UNSUPPORTED), (dict(r=-8), g.ERR_SHAPE), (dict(r=12), g.ERR_UNSUPPORTED),
    (dict(r=264), g.ERR_UNSUPPORTED), (dict(d=16512, mods=[module(k_in=16512)]), g.ERR_UNSUPPORTED), (dict(x=None), g.ERR_INVALID_ARG),
    (dict(off=None), g.ERR_INVALID_ARG), (dict(tok=None), g.ERR_SHAPE), (dict(b=None), g.ERR_INVALID_ARG), (dict(mods=[module(a=None)]), g.ERR_INVALID_ARG),
    (dict(mods=[module(q=None)]), g.ERR_INVALID_ARG), (dict(mods=[module(sz=None)]), g.ERR_INVALID_ARG), (dict(mods=[module(y=None)]), g.ERR_INVALID_ARG),
    (dict(mods=[module(k_in=384)]), g.ERR_SHAPE), (dict(mods=[module(n_out=0)]), g.ERR_SHAPE), (dict(mods=[module(q=FAKE + 8)]), g.ERR_ALIGN),
    (dict(mods=[module(y=FAKE + 2)]), g.ERR_ALIGN), (dict(x=FAKE + 2), g.ERR_ALIGN), (dict(b=FAKE + 8), g.ERR_ALIGN), (dict(off=FAKE + 2), g.ERR_ALIGN),
    (dict(tok=FAKE + 1), g.ERR_ALIGN), (dict(ws=None), g.ERR_WORKSPACE), (dict(n=HDR), g.ERR_WORKSPACE), (dict(ws=FAKE + 16), g.ERR_ALIGN),
    (dict(n_rows=1 << 23, mods=[module(n_out=1 << 24)] * 4, n=1 << 40), g.ERR_UNSUPPORTED), (dict(n_rows=0), g.OK),
])
def test_experts_refusals(kw, status):
    assert experts(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), g.ERR_INVALID_ARG), (dict(scales=None), g.ERR_INVALID_ARG), (dict(q=None), g.ERR_INVALID_ARG),
    (dict(sz=None), g.ERR_INVALID_ARG), (dict(flag=None), g.ERR_INVALID_ARG), (dict(k=96), g.ERR_SHAPE), (dict(n=0), g.ERR_SHAPE),
    (dict(codes=FAKE + 8), g.ERR_ALIGN), (dict(q=FAKE + 8), g.ERR_ALIGN), (dict(scales=FAKE + 2), g.ERR_ALIGN),
])
def test_repack_refusals(kw, status):
    a = dict(codes=FAKE, scales=FAKE, n=16, k=128, q=FAKE, sz=FAKE, flag=FAKE)
    a.update(kw)
    assert g.lib().glowq_repack_fp8(a["codes"], a["scales"], a["n"], a["k"], a["q"], a["sz"], a["flag"], None) == status
