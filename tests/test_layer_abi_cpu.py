"""The 8-bit integer group forward, the routed-row calls and the gated activation without a GPU:
sizes, and every refusal before any HIP call."""
import ctypes

import pytest
import torch

from rank_error_compensation_amd import glowq as g

FAKE = 0x10000   # aligned fake device address: never dereferenced, validation fails first
HDR = 8192


def r256(n):
    return (n + 255) // 256 * 256


def test_w8_sizes():
    L = g.lib()
    assert L.glowq_w8_q_bytes(4096, 4096) == 4096 * 4096
    assert L.glowq_w8_q_bytes(17, 256) == 2 * 16 * 256   # rows padded to 32
    assert L.glowq_w8_sz_bytes(17) == 2 * 64
    for n, k in ((0, 128), (16, 100), (16, 0), (16, 16384 + 128), ((1 << 24) + 1, 128), (-1, 128)):
        assert L.glowq_w8_q_bytes(n, k) == 0
    assert L.glowq_w8_sz_bytes(0) == 0 and L.glowq_w8_sz_bytes((1 << 24) + 1) == 0


def test_w8a8_workspace_bytes():
    f = g.lib().glowq_w8a8_workspace_bytes
    assert f(3, 256, 0) >= r256(3 * 256) + r256(12)
    assert f(3, 256, 64) > f(3, 256, 0)
    for T, d, r in ((0, 256, 0), (-1, 256, 0), (3, 100, 0), (3, 16384 + 128, 0), (3, 256, -8), (3, 256, 264),
                    ((1 << 20) + 1, 128, 0)):
        assert f(T, d, r) == 0
    # a workspace for the largest call serves every smaller one
    Ts = [1, 2, 16, 31, 32, 33, 63, 64, 65, 100, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049, 3000, 8191, 8193, 65536]
    for d in (128, 2048, 4096, 11008, 16384):
        for r in (0, 8, 64, 72, 256):
            n = [f(T, d, r) for T in Ts]
            assert n == sorted(n), (d, r)
            assert r == 256 or all(f(T, d, r) <= f(T, d, r + 8) for T in Ts)
            assert d == 16384 or all(f(T, d, r) <= f(T, d + 128, r) for T in Ts)


def w8(fmt=4, n_out=32, k_in=256, q=FAKE, sz=FAKE, reserved=0):
    return g.QWeightC(q, sz, n_out, k_in, fmt, reserved)


def forward(x=FAKE, T=4, d=256, w=None, m=None, b=FAKE, a=FAKE, r=8, restore=1, ws=FAKE, n=1 << 30, y=FAKE):
    w = [w8()] if w is None else w
    m = len(w) if m is None else m
    wc = (g.QWeightC * max(1, len(w)))(*w)
    ac = (ctypes.c_void_p * max(1, len(w)))(*([a] * max(1, len(w))))
    yc = (ctypes.c_void_p * max(1, len(w)))(*([y] * max(1, len(w))))
    return g.lib().glowq_group_forward_w8a8(x, T, d, m, wc, b, ac, r, restore, ws, n, yc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), g.ERR_INVALID_ARG), (dict(y=None), g.ERR_INVALID_ARG), (dict(a=None), g.ERR_INVALID_ARG),
    (dict(b=None), g.ERR_INVALID_ARG), (dict(w=[w8(q=None)]), g.ERR_INVALID_ARG),
    (dict(w=[w8(sz=None)]), g.ERR_INVALID_ARG), (dict(w=[w8(fmt=5)]), g.ERR_INVALID_ARG),
    (dict(w=[w8(fmt=-1)]), g.ERR_INVALID_ARG), (dict(w=[w8(reserved=1)]), g.ERR_INVALID_ARG),
    (dict(w=[w8(fmt=0)]), g.ERR_UNSUPPORTED), (dict(w=[w8(fmt=1)]), g.ERR_UNSUPPORTED),
    (dict(w=[w8(), w8(fmt=0)]), g.ERR_UNSUPPORTED), (dict(w=[w8()] * 8, m=9), g.ERR_UNSUPPORTED),
    (dict(m=0), g.ERR_SHAPE), (dict(T=-1), g.ERR_SHAPE), (dict(d=100), g.ERR_SHAPE), (dict(d=0), g.ERR_SHAPE),
    (dict(w=[w8(k_in=128)]), g.ERR_SHAPE), (dict(w=[w8(n_out=0)]), g.ERR_SHAPE), (dict(r=-8), g.ERR_SHAPE),
    (dict(r=12), g.ERR_UNSUPPORTED), (dict(r=264), g.ERR_UNSUPPORTED),
    (dict(d=16512, w=[w8(k_in=16512)]), g.ERR_UNSUPPORTED),
    (dict(T=1 << 20, d=2048, w=[w8(k_in=2048)]), g.ERR_UNSUPPORTED),
    (dict(x=FAKE + 8), g.ERR_ALIGN), (dict(y=FAKE + 8), g.ERR_ALIGN), (dict(b=FAKE + 8), g.ERR_ALIGN),
    (dict(a=FAKE + 8), g.ERR_ALIGN), (dict(w=[w8(q=FAKE + 4)]), g.ERR_ALIGN), (dict(ws=FAKE + 16), g.ERR_ALIGN),
    (dict(ws=None), g.ERR_WORKSPACE), (dict(n=64), g.ERR_WORKSPACE), (dict(restore=0, n=64), g.ERR_WORKSPACE),
    (dict(T=0), g.OK),
])
def test_w8a8_refusals(kw, status):
    assert forward(**kw) == status


def test_other_forwards_refuse_int8_weights():
    L = g.lib()
    wc = (g.QWeightC * 1)(w8())
    p = (ctypes.c_void_p * 1)(FAKE)
    assert L.glowq_group_forward(FAKE, 4, 256, 1, wc, FAKE, p, 8, 1, FAKE, 1 << 24, p, None) == g.ERR_INVALID_ARG
    assert L.glowq_dequant(ctypes.byref(wc[0]), FAKE, 0, None) == g.ERR_INVALID_ARG


def test_every_other_entry_point_refuses_int8_weights():
    L, big = g.lib(), 1 << 30
    wc = (g.QWeightC * 1)(w8())
    p = (ctypes.c_void_p * 1)(FAKE)
    unit = (g.UnitC * 1)(g.UnitC(1, 1, FAKE, 4, 256, wc, FAKE, p, 8, 1, p))
    for r in (0, 8):
        assert L.glowq_solo_forward(FAKE, 4, 256, wc, FAKE, FAKE, r, 1, FAKE, big, FAKE, None) == g.ERR_INVALID_ARG
        assert L.glowq_group_forward_static(FAKE, 4, 256, 1, wc, FAKE, p, r, 1, p, None) == g.ERR_INVALID_ARG
        for f in (L.glowq_group_forward_w4a8, L.glowq_group_forward_mx8):
            assert f(FAKE, 4, 256, 1, wc, FAKE, p, r, 1, FAKE, big, p, None) == g.ERR_INVALID_ARG
        assert L.glowq_layerwise_forward(FAKE, 4, 256, 1, wc, p, p, r, 1, FAKE, big, p, None) == g.ERR_INVALID_ARG
    assert L.glowq_path_forward(unit, 1, FAKE, big, None) == g.ERR_INVALID_ARG
    assert L.glowq_ner_sums(FAKE, wc, FAKE, big, FAKE, None) == g.ERR_UNSUPPORTED
    wp = ctypes.cast(p, ctypes.POINTER(ctypes.c_void_p))
    assert L.glowq_ner_sums_batch(1, wp, wc, FAKE, big, FAKE, None) == g.ERR_UNSUPPORTED


def host_weight(fmt, n_out=32, k_in=256):
    """A weight with buffers of its format's sizes (the experts' product takes INT4 alone)."""
    L = g.lib()
    if fmt == g.FMT_INT8_CHANNEL:
        q, z = L.glowq_w8_q_bytes(n_out, k_in), L.glowq_w8_sz_bytes(n_out)
    else:
        q, z = L.glowq_q_bytes(n_out, k_in), L.glowq_sz_bytes(n_out, k_in)
    return g.QWeight(torch.zeros(q, dtype=torch.uint8), torch.zeros(z, dtype=torch.uint8), n_out, k_in, fmt)


@pytest.mark.parametrize("fmts", [[g.FMT_INT8_CHANNEL] * 2, [g.FMT_INT4_G128, g.FMT_INT8_CHANNEL],
                                  [g.FMT_MXFP4] * 2, [g.FMT_MXFP6_E2M3], [g.FMT_INT4_G128, g.FMT_MXFP6_E3M2]])
def test_stacked_experts_refuse_other_formats(fmts):
    with pytest.raises(g.GlowQError) as e:
        g.MoeModule.stack([host_weight(f) for f in fmts], None)
    assert e.value.status == g.ERR_UNSUPPORTED


def test_stacked_experts_refuse_mixed_shapes_and_none():
    for ws in ([], [host_weight(0), host_weight(0, 48)], [host_weight(0), host_weight(0, 32, 384)]):
        with pytest.raises(g.GlowQError) as e:
            g.MoeModule.stack(ws, None)
        assert e.value.status == g.ERR_SHAPE
    m = g.MoeModule.stack([host_weight(0), host_weight(0)], None)
    assert m.n_out == 32 and m.k_in == 256 and m.q.numel() == 2 * g.lib().glowq_q_bytes(32, 256)


@pytest.mark.parametrize("n_out,k_in,n_exp", [(1, 128, 1), (17, 256, 3), (1408, 2048, 2)])
def test_moe_forward_takes_modules_of_exactly_their_experts(n_out, k_in, n_exp):
    """Buffers of the library's own sizes pass (a call without rows: nothing is launched)."""
    m = g.MoeModule.stack([host_weight(0, n_out, k_in)] * n_exp, None)
    x, off = torch.zeros(0, k_in, dtype=torch.float16), torch.zeros(n_exp + 1, dtype=torch.int32)
    ys = g.moe_forward(x, n_exp, [m], None, g.MOE_SHARE_EXPERT, 0, False, None, off, 0,
                       workspace=torch.zeros(HDR, dtype=torch.uint8), stream=type("S", (), {"cuda_stream": 0}))
    assert ys[0].shape == (0, n_out)


@pytest.mark.parametrize("case", ["int8 scales", "short codes", "fewer experts"])
def test_moe_forward_refuses_modules_smaller_than_their_experts(case):
    """Buffers that do not hold n_exp INT4 modules are never handed to the kernels."""
    m = g.MoeModule.stack([host_weight(0), host_weight(0)], None)
    if case == "int8 scales":
        w = host_weight(g.FMT_INT8_CHANNEL)
        m = g.MoeModule(torch.cat([w.q, w.q]), torch.cat([w.sz, w.sz]), None, 32, 256)
    elif case == "short codes":
        m = g.MoeModule(m.q[:-1], m.sz, None, 32, 256)
    x, off = torch.zeros(2, 256, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(g.GlowQError) as e:
        g.moe_forward(x, 3 if case == "fewer experts" else 2, [m], None, g.MOE_SHARE_EXPERT, 0, False, None, off, 2,
                      workspace=torch.zeros(HDR, dtype=torch.uint8), stream=type("S", (), {"cuda_stream": 0}))
    assert e.value.status == g.ERR_SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), g.ERR_INVALID_ARG), (dict(scales=None), g.ERR_INVALID_ARG), (dict(flag=None), g.ERR_INVALID_ARG),
    (dict(n=0), g.ERR_SHAPE), (dict(k=100), g.ERR_SHAPE), (dict(k=16512), g.ERR_UNSUPPORTED),
    (dict(n=(1 << 24) + 1), g.ERR_UNSUPPORTED), (dict(codes=FAKE + 4), g.ERR_ALIGN), (dict(scales=FAKE + 2), g.ERR_ALIGN),
])
def test_repack_w8_refusals(kw, status):
    a = dict(codes=FAKE, scales=FAKE, n=16, k=128, flag=FAKE)
    a.update(kw)
    assert g.lib().glowq_repack_w8(a["codes"], a["scales"], a["n"], a["k"], FAKE, FAKE, a["flag"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), g.ERR_SHAPE), (dict(k=0), g.ERR_SHAPE), (dict(k=65), g.ERR_UNSUPPORTED),
    (dict(E=0), g.ERR_UNSUPPORTED), (dict(E=257), g.ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), g.ERR_UNSUPPORTED),
    (dict(T=1 << 20, k=9), g.ERR_UNSUPPORTED), (dict(ids=None), g.ERR_INVALID_ARG), (dict(off=None), g.ERR_INVALID_ARG),
    (dict(tok=None), g.ERR_INVALID_ARG), (dict(pr=None), g.ERR_INVALID_ARG), (dict(ids=FAKE + 2), g.ERR_ALIGN),
    (dict(ws=None), g.ERR_WORKSPACE), (dict(n=HDR - 1), g.ERR_WORKSPACE), (dict(T=100000, n=HDR), g.ERR_WORKSPACE),
    (dict(ws=FAKE + 128), g.ERR_ALIGN),
])
def test_moe_sort_refusals(kw, status):
    a = dict(ids=FAKE, T=4, k=2, E=8, off=FAKE, tok=FAKE, pr=FAKE, ws=FAKE, n=HDR)
    a.update(kw)
    assert g.lib().glowq_moe_sort(a["ids"], a["T"], a["k"], a["E"], a["off"], a["tok"], a["pr"], a["ws"], a["n"],
                                  None) == status


def test_moe_sort_workspace():
    f = g.lib().glowq_moe_sort_workspace_bytes
    assert f(0, 4, 60) == HDR and f(1, 4, 60) == HDR
    assert f(1 << 20, 8, 256) > HDR
    for T, k, E in ((-1, 4, 60), (4, 0, 60), (4, 65, 60), (4, 4, 0), (4, 4, 257), (1 << 20, 9, 60)):
        assert f(T, k, E) == 0


ROWS = [(dict(dtype=2), g.ERR_INVALID_ARG), (dict(d=0), g.ERR_SHAPE), (dict(T=-1), g.ERR_SHAPE),
        (dict(n_rows=-1), g.ERR_SHAPE), (dict(d=(1 << 20) + 1), g.ERR_UNSUPPORTED),
        (dict(n_rows=(1 << 23) + 1), g.ERR_UNSUPPORTED), (dict(x=None), g.ERR_INVALID_ARG),
        (dict(out=None), g.ERR_INVALID_ARG), (dict(lst=None), g.ERR_INVALID_ARG), (dict(x=FAKE + 8), g.ERR_ALIGN),
        (dict(out=FAKE + 4), g.ERR_ALIGN), (dict(lst=FAKE + 1), g.ERR_ALIGN), (dict(ws=None), g.ERR_WORKSPACE),
        (dict(n=HDR - 256), g.ERR_WORKSPACE), (dict(ws=FAKE + 64), g.ERR_ALIGN)]


def rows_args(kw):
    a = dict(x=FAKE, T=4, d=16, dtype=1, lst=FAKE, n_rows=8, out=FAKE, ws=FAKE, n=HDR, k=2, w=FAKE, add=None, tok=FAKE,
             rows=FAKE, dw=FAKE)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", ROWS + [(dict(T=0, lst=None), g.ERR_INVALID_ARG), (dict(n_rows=0, x=None), g.OK)])
def test_moe_dispatch_refusals(kw, status):
    a = rows_args(kw)
    assert g.lib().glowq_moe_dispatch(a["x"], a["T"], a["d"], a["dtype"], a["lst"], a["n_rows"], a["out"], a["ws"],
                                      a["n"], None) == status


@pytest.mark.parametrize("kw,status", ROWS + [(dict(T=0, x=None), g.OK), (dict(k=0), g.ERR_SHAPE),
                                              (dict(k=65), g.ERR_UNSUPPORTED), (dict(w=FAKE + 2), g.ERR_ALIGN),
                                              (dict(add=FAKE + 8), g.ERR_ALIGN)])
def test_moe_combine_refusals(kw, status):
    a = rows_args(kw)
    assert g.lib().glowq_moe_combine(a["x"], a["n_rows"], a["lst"], a["w"], a["add"], a["T"], a["k"], a["d"], a["dtype"],
                                     a["out"], a["ws"], a["n"], None) == status


@pytest.mark.parametrize("kw,status", ROWS + [(dict(T=0, n_rows=0, x=None), g.OK), (dict(k=0), g.ERR_SHAPE),
                                              (dict(T=0, out=None), g.ERR_INVALID_ARG), (dict(tok=None), g.ERR_INVALID_ARG), (dict(rows=None), g.ERR_INVALID_ARG),
                                              (dict(dw=None), g.ERR_INVALID_ARG), (dict(dw=FAKE + 2), g.ERR_ALIGN),
                                              (dict(rows=FAKE + 8), g.ERR_ALIGN)])
def test_moe_combine_backward_refusals(kw, status):
    a = rows_args(kw)
    assert g.lib().glowq_moe_combine_backward(a["x"], a["rows"], a["n_rows"], a["lst"], a["tok"], a["w"], a["T"], a["k"],
                                              a["d"], a["dtype"], a["out"], a["dw"], a["ws"], a["n"], None) == status


@pytest.mark.parametrize("kw,status", ROWS + [(dict(T=0, n_rows=0, x=None), g.OK), (dict(k=0), g.ERR_SHAPE),
                                              (dict(T=0, out=None), g.ERR_INVALID_ARG), (dict(tok=None), g.ERR_INVALID_ARG), (dict(rows=None), g.ERR_INVALID_ARG),
                                              (dict(dw=None), g.ERR_INVALID_ARG), (dict(dw=FAKE + 2), g.ERR_ALIGN),
                                              (dict(x=FAKE + 32, out=FAKE), g.ERR_INVALID_ARG)])
def test_moe_combine_backward_whole_refusals(kw, status):
    a = rows_args(kw)
    assert g.lib().glowq_moe_combine_backward_whole(a["x"], a["rows"], a["n_rows"], a["lst"], a["tok"], a["w"], a["T"],
                                                    a["k"], a["d"], a["dtype"], a["out"], a["dw"], a["ws"], a["n"],
                                                    None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), g.ERR_INVALID_ARG), (dict(n=-1), g.ERR_SHAPE), (dict(n=(1 << 33) + 1), g.ERR_UNSUPPORTED),
    (dict(gate=None), g.ERR_INVALID_ARG), (dict(up=None), g.ERR_INVALID_ARG), (dict(h=None), g.ERR_INVALID_ARG),
    (dict(gate=FAKE + 8), g.ERR_ALIGN), (dict(h=FAKE + 2), g.ERR_ALIGN), (dict(n=0, gate=None), g.OK)])
def test_swiglu_refusals(kw, status):
    a = dict(gate=FAKE, up=FAKE, n=8, dtype=1, h=FAKE)
    a.update(kw)
    L = g.lib()
    assert L.glowq_swiglu(a["gate"], a["up"], a["n"], a["dtype"], a["h"], None) == status
    assert L.glowq_swiglu_backward(FAKE, a["gate"], a["up"], a["n"], a["dtype"], a["h"], FAKE, None) == status
    if a["n"]:
        assert L.glowq_swiglu_backward(None, FAKE, FAKE, 8, 1, FAKE, FAKE, None) == g.ERR_INVALID_ARG
        assert L.glowq_swiglu_backward(FAKE, FAKE, FAKE, 8, 1, FAKE, None, None) == g.ERR_INVALID_ARG


FAR = [FAKE + (i << 20) for i in range(8)]  # addresses with room between them


def test_overlapping_tensors_are_refused():
    L, bad = g.lib(), g.ERR_INVALID_ARG
    a, b, c, o, tok, ws, w, e = FAR
    row = 16 * 2  # fp16 rows of 16 values
    for x in (o, o + 7 * row, o - 3 * row):
        assert L.glowq_moe_dispatch(x, 4, 16, 1, tok, 8, o, ws, HDR, None) == bad
    for rows, add in ((o, None), (o - 7 * row, b), (a, o + row), (a, o - 3 * row)):
        assert L.glowq_moe_combine(rows, 8, c, w, add, 4, 2, 16, 1, o, ws, HDR, None) == bad
    for dy, rows in ((o, a), (o + 7 * row, a), (a, o + row), (a, o - row)):
        assert L.glowq_moe_combine_backward(dy, rows, 8, c, tok, w, 4, 2, 16, 1, o, e, ws, HDR, None) == bad
    for ids, off, t, p in ((a, b, a, o), (a, b, c, a + 28), (a, a + 28, c, o), (a, b, c, c + 16), (a, o + 4, c, o)):
        assert L.glowq_moe_sort(ids, 4, 2, 3, off, t, p, ws, HDR, None) == bad
    assert L.glowq_swiglu(a, b, 64, 1, a + 16, None) == bad and L.glowq_swiglu(a, b, 64, 1, b - 112, None) == bad
    for dg, du in ((a + 16, o), (o, b + 16), (c - 112, o), (o, o), (o, o + 16)):
        assert L.glowq_swiglu_backward(a, b, c, 64, 1, dg, du, None) == bad


def test_python_checks_refuse_host_tensors():
    x = torch.zeros(2, 16)
    i = torch.zeros(2, 2, dtype=torch.int32)
    calls = [lambda: g.swiglu(x, x), lambda: g.swiglu_backward(x, x, x), lambda: g.moe_sort(i, 4),
             lambda: g.moe_dispatch(x, i.view(-1)), lambda: g.moe_combine(x, i, None),
             lambda: g.moe_combine_backward(x, x, i, torch.zeros(2, dtype=torch.int32), None),
             lambda: g.group_forward_w8a8(x.half(), [], None, [], 0, False)]
    for f in calls:
        with pytest.raises(g.GlowQError) as e:
            f()
        assert e.value.status == g.ERR_INVALID_ARG


@pytest.mark.parametrize("f", [
    lambda x, i: g.swiglu(x, x.half()), lambda x, i: g.swiglu(x, x[:1]), lambda x, i: g.swiglu(x.double(), x.double()),
    lambda x, i: g.moe_sort(i.long(), 4), lambda x, i: g.moe_sort(i.view(-1), 4),
    lambda x, i: g.moe_dispatch(x.bfloat16(), i.view(-1)), lambda x, i: g.moe_dispatch(x, i),
    lambda x, i: g.moe_combine(x, i, torch.zeros(2, 2, dtype=torch.float16)),
    lambda x, i: g.moe_combine(x, i, torch.zeros(2, 3)),
    lambda x, i: g.QWeight.from_int8(torch.zeros(4, 128), torch.zeros(4)),
    lambda x, i: g.QWeight.from_int8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(5)),
])
def test_python_checks_refuse_types_and_shapes(f):
    with pytest.raises(g.GlowQError) as e:
        f(torch.zeros(2, 16), torch.zeros(2, 2, dtype=torch.int32))
    assert e.value.status in (g.ERR_INVALID_ARG, g.ERR_SHAPE)


def test_routing_status_has_its_name():
    assert g.lib().glowq_status_string(g.ERR_ROUTING).startswith(b"GLOWQ_ERR_ROUTING")
    assert "GLOWQ_ERR_ROUTING" in str(g.GlowQError(g.ERR_ROUTING, "glowq_moe_sort"))


def test_from_int8_refuses_a_stream_of_another_device():
    """The repack would run on one device with the other's memory."""
    stream = type("S", (), {"device": torch.device("cuda:1"), "cuda_stream": 0})
    codes, scales = torch.zeros(16, 128, dtype=torch.int8), torch.ones(16)
    for device in ("cuda:0", torch.device("cuda", 0)):
        with pytest.raises(g.GlowQError) as e:
            g.QWeight.from_int8(codes, scales, device=device, stream=stream)
        assert e.value.status == g.ERR_INVALID_ARG
