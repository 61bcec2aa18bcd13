"""64-bit reference forms of the 8-bit float layers and of the heads' pass, and the error bounds the GPU tests hold them to,
in numpy."""
from __future__ import annotations

import numpy as np

from q8ref import E, half_ulp, widen  # noqa: F401

BLOCK, TOP = 128, 448.0


def e4m3(v):
    """The nearest e4m3 value, ties to even, within +-448: steps of 2^(e - 3) from 2^e on, of 2^-9 below 2^-6."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(a)) - 3)
    return np.clip(np.rint(v / step) * step, -TOP, TOP)


def decode(q):
    """The values that e4m3 bytes stand for."""
    q = q.astype(np.int64)
    sign, e, m = np.where(q & 128, -1.0, 1.0), (q >> 3) & 15, q & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where((q & 127) == 127, np.nan, sign * v)


def blocks(n):
    return -(-n // BLOCK)


def quantize(x64, rows=1):
    """(values, scales) of x whose values fp32 holds exactly, blocks of `rows` x 128; scales [row blocks, column blocks].
    The scale and the quotient are fp32 by definition."""
    x = x64.astype(np.float32)
    m, k = x.shape
    q = np.zeros((m, k))
    s = np.zeros((-(-m // rows), blocks(k)), np.float32)
    with np.errstate(all="ignore"):
        for r in range(s.shape[0]):
            for c in range(s.shape[1]):
                b = x[r * rows:(r + 1) * rows, c * BLOCK:(c + 1) * BLOCK]
                if not np.isfinite(b).all():
                    s[r, c] = np.nan
                    continue
                s[r, c] = np.abs(b).max() / np.float32(TOP)
                if s[r, c] > 0:
                    q[r * rows:(r + 1) * rows, c * BLOCK:(c + 1) * BLOCK] = e4m3(
                        np.clip((b / s[r, c]).astype(np.float32).astype(np.float64), -TOP, TOP))
    return q, s


def spread(s, n, k, rows):
    """Scales [row blocks, column blocks] for each value."""
    return np.repeat(np.repeat(s.astype(np.float64), rows, axis=0)[:n], BLOCK, axis=1)[:, :k]


def product(x, w, bias=None, dx=None, narrow=False):
    """(y, error bound) of x w^T (+ bias) for tokens and weights in values (q s), from tokens with error dx.

    A block's 128 products are exact in fp32 (two 4-bit fractions); its sum is held to 128 roundings of one step each
    (a sum that truncates is off by a whole one, 2 E), of the block's sum of magnitudes; then comes one rounding of the two
    scales' product, and one for each block's addition; 16 more join the parts of a K that is cut, and one adds the bias.

    narrow (16-bit outputs): the 8-bit matrix instruction first cuts groups of 8 products at 2^-13 of the power of two of
    the largest: each of them loses less than that, the 8 together 2^-10 of it, and a group's largest product is at most its
    sum of magnitudes."""
    y = x @ w.T
    a = np.abs(x) @ np.abs(w).T
    d = ((2 * 128 + blocks(x.shape[1]) + 20) * E + (2.0 ** -10 if narrow else 0)) * a + 1e-37
    if dx is not None:
        d = d + dx @ np.abs(w).T
    if bias is not None:
        y = y + bias
        d = d + E * np.abs(y)
    return y, d


def gate(g, dg, u, du):
    """(silu(g) u, error bound)."""
    with np.errstate(over="ignore"):
        a = g / (1 + np.exp(-g))
    # silu' is at most 1.1; exp is good to 2 ulp, then one addition, one division and two products
    return a * u, 1.1 * dg * np.abs(u) + np.abs(a) * du + 1.1 * dg * du + 8 * E * np.abs(a * u) + 1e-36 * np.abs(u)


def cut(h, dh):
    """(values, error bound) of rows h, known to dh, cut to e4m3 in blocks of 128 columns: rounding is monotone, so the
    values lie between those of h - dh and h + dh; a block's scale, and the quotient with it, is off by its largest value's
    relative error and two roundings."""
    v, d = np.zeros_like(h), np.zeros_like(h)
    for c in range(0, h.shape[1], BLOCK):
        b, db = h[:, c:c + BLOCK], dh[:, c:c + BLOCK]
        top = np.abs(b).max(axis=1, keepdims=True)
        rel = np.where(top > 0, db.max(axis=1, keepdims=True) / np.maximum(top, 1e-300), 0) + 2 * E
        s = np.maximum(top / TOP, 1e-300)
        at = lambda x: e4m3(np.clip(x / s, -TOP, TOP)) * s
        off = db + 3 * rel * np.abs(b)
        v[:, c:c + BLOCK] = at(b)
        d[:, c:c + BLOCK] = np.maximum(at(b + off) - at(b), at(b) - at(b - off)) + 2 * rel * np.abs(at(b))
    return v, d


def check(got, ref, bound, out):
    """Every value within its bound plus half an ulp of the output type."""
    got = widen(got) if not isinstance(got, np.ndarray) else got.astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.isfinite(got).all()
    off = np.abs(got - ref) - bound - half_ulp(ref, out) * (1 + 1e-6)
    worst = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert off.size == 0 or off[worst] <= 0, "at %s: %r, expected %r within %g" % (
        worst, got[worst], ref[worst], bound[worst] if np.ndim(bound) else bound)


# ------------------------------------------------------------------ heads

def rotate(x, pos, freqs, rot, start=0, interleaved=False, scale=1.0, norm="none", w=None, b=None, eps=1e-6, w_offset=0.0):
    """(y, error bound): x [batch, tokens, heads, dim], pos [batch, tokens], freqs in radians per position.

    Norm: a sum of up to 1024 squares passes at most 32 + 6 roundings (32 values of a lane, 6 steps over the lanes), half of
    which the square root leaves; the mean the same.  Sines: the angle's fp32 part is at most pi / 4 off by half an ulp, 0.4 E
    as an angle, and the functions are good to 2 ulp: 3 E with the scale's product; then one product and one fused step."""
    f = lambda v: np.float64(np.float32(v))
    y, d = x.astype(np.float64), np.zeros(x.shape)
    if norm != "none":
        if norm == "layer":
            mean = y.mean(axis=-1, keepdims=True)
            d = d + 40 * E * np.abs(y).mean(axis=-1, keepdims=True) + E * np.abs(y - mean)
            y = y - mean
        sig = np.sqrt((y ** 2).mean(axis=-1, keepdims=True) + f(eps))
        rel = 24 * E + np.sqrt((d ** 2).mean(axis=-1, keepdims=True)) / sig
        k = 1.0 if w is None else f(w_offset) + w
        y, d = y / sig * k, np.abs(k) / sig * d + np.abs(y / sig * k) * (rel + 4 * E)
        if b is not None:
            y, d = y + b, d + E * np.abs(y + b)
    if rot:
        j = np.arange(rot // 2)
        i0 = start + (2 * j if interleaved else j)
        i1 = i0 + (1 if interleaved else rot // 2)
        ang = (pos.astype(np.float64)[..., None] * np.asarray(freqs, np.float64))[:, :, None]
        c, s = np.cos(ang) * f(scale), np.sin(ang) * f(scale)
        p, q, dp, dq = y[..., i0], y[..., i1], d[..., i0], d[..., i1]
        amp = abs(f(scale)) * (np.abs(p) + np.abs(q))
        y, d = y.copy(), d.copy()
        y[..., i0], y[..., i1] = p * c - q * s, p * s + q * c
        # fp64 angles of far positions are off by the product's rounding themselves, here and there
        ferr = 4 * np.abs(ang) * 2.0 ** -53
        d[..., i0] = np.abs(c) * dp + np.abs(s) * dq + amp * (5 * E + ferr)
        d[..., i1] = np.abs(s) * dp + np.abs(c) * dq + amp * (5 * E + ferr)
    return y, d + 1e-37
