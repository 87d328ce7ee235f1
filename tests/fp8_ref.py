"""Plain fp64 reference (numpy) of the block-scaled e4m3 products, with elementwise error bounds from eps / 2 of each
type."""
import numpy as np

from layer_ref import HALF, TINY, U32, f64


def e4m3_round(v):
    """Nearest e4m3 number of fp32 values |v| <= 464 (ties to even), by the format's steps: 2^(e - 3) for 2^e <= |v| <
    2^(e + 1), e >= -6."""
    a = np.abs(v.astype(np.float64))
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)
    return np.copysign(np.round(a / step) * step, v)


def e4m3_bytes(v):
    """Codes of e4m3 numbers."""
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -30)))
    normal = e >= -6
    mant = np.where(normal, a / np.exp2(np.maximum(e, -6.0)) - 1.0, a / 2.0 ** -6) * 8
    code = np.where(normal, (e + 7) * 8, 0) + mant
    return (code + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantise(x):
    """(codes as numbers [T][d], scales fp32 [T][d / 128]) of fp16 x; fp32 steps as documented."""
    v = x.detach().cpu().float().numpy()
    T, d = v.shape
    v = v.reshape(T, d // 128, 128)
    top = np.abs(v).max(2)
    with np.errstate(divide="ignore", invalid="ignore"):
        scale = (top / np.float32(448)).astype(np.float32)
        inv = np.where(top > 0, np.float32(448) / top, np.float32(0)).astype(np.float32)
        u = (v * inv[:, :, None]).astype(np.float32)
    return e4m3_round(u).reshape(T, d), scale


def product(x, q, scales, b, a, correct):
    """(y, bound) of one module: q e4m3 [n][d], scales [ceil(n / 128)][d / 128].  Bound: a group's 128 products in the
    matrix core, its scaling (three steps) and the sum over the groups in any order; R's fp32 sum over d and its
    rounding to fp16, the fp32 sum over r, the final rounding.
    The matrix core brings eight products at a time (eight consecutive inputs) to the exponent of the largest, 2^e, and
    drops what lies below 2^(e - 13): beside a product of 2^16 one of 2^3 counts whole and one of 2^2 not at all,
    whatever its sign, while products of other eights lose nothing but fp32's roundings (measured with single products in
    all places).  The largest product itself is a multiple of 2^(e - 6), so at most seven lose less than 2^(e - 13) each:
    7 2^-13 2^e, and 2^e <= the largest |c| times the largest |q| of the eight; the sixteen sums then meet in fp32."""
    c, s = quantise(x)
    T, d = c.shape
    qf = q.detach().cpu().float().double().numpy()
    n, G = qf.shape[0], d // 128
    S = f64(scales)[np.arange(n) // 128]
    y, mag, most, drop = np.zeros((T, n)), np.zeros((T, n)), np.zeros((T, n)), np.zeros((T, n))
    c8, q8 = np.abs(c).reshape(T, G, 16, 8).max(3), np.abs(qf).reshape(n, G, 16, 8).max(3)
    for g in range(G):
        k = slice(128 * g, 128 * g + 128)
        w = s[:, g, None].astype(np.float64) * S[None, :, g]
        y += w * (c[:, k] @ qf[:, k].T)
        mag += np.abs(w) * (np.abs(c[:, k]) @ np.abs(qf[:, k]).T)
        most += np.abs(w * (c[:, k] @ qf[:, k].T))
        drop += np.abs(w) * (c8[:, g] @ q8[:, g].T)
    err = (7 * 2.0 ** -13 * drop + U32 * (128 * mag + (G + 4) * most)) * 1.01
    if correct:
        xf, bf, af = f64(x), f64(b), f64(a)
        R = xf @ bf.T
        r = bf.shape[0]
        dR = d * U32 * (np.abs(xf) @ np.abs(bf).T) * 1.01 + HALF["f16"] * np.abs(R) + TINY["f16"]
        corr = R @ af.T
        y = y + corr
        err = err + dR @ np.abs(af).T * 1.01 + (r + 1) * U32 * (np.abs(R) @ np.abs(af).T + np.abs(y)) * 1.01
    return y, err * 1.01 + HALF["f16"] * (np.abs(y) + err) + TINY["f16"]
