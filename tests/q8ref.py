"""64-bit reference forms of the 8-bit operators and the error bounds the GPU tests hold them to, in numpy."""
from __future__ import annotations

import numpy as np

E = 2.0 ** -24  # half an ulp of fp32, relative


def widen(t) -> np.ndarray:
    """A device or host tensor of any float type as float64."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def half_ulp(ref, out: str):
    """Half a unit in the last place of the output type at |ref|."""
    mant, emin = {"f16": (10, -14), "bf16": (7, -126), "f32": (23, -126)}[out]
    a = np.maximum(np.abs(ref), 2.0 ** emin)
    return 0.5 * np.exp2(np.floor(np.log2(a)) - mant)


def quantize(x64):
    """(q, s) of rows whose values fp32 holds exactly: s and the quotient are fp32 by definition."""
    x = x64.astype(np.float32)
    with np.errstate(all="ignore"):
        s = (np.abs(x).max(axis=1) / np.float32(127)).astype(np.float32)
        bad = ~np.isfinite(x).all(axis=1)
        s[bad] = np.nan
        den = np.where((s > 0) & ~bad, s, np.float32(1))[:, None]
        q = np.rint((x / den).astype(np.float32))
        q = np.where((s > 0)[:, None] & ~bad[:, None], np.clip(q, -127, 127), 0)
    return q.astype(np.int8), s


def product(q, s, w, sw, bias=None):
    """(y, error bound) of the scaled product: one rounding of the exact sum to fp32, two products, one addition."""
    t = (q.astype(np.float64) @ w.astype(np.float64).T) * s.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    b = 0.0 if bias is None else bias.astype(np.float64)[None, :]
    return t + b, 3 * E * np.abs(t) + (0 if bias is None else E * np.abs(t + b)) + 1e-37


def gated(q, s, w, sw, bias=None):
    """(silu(g) u, error bound), g and u the two halves of w's rows."""
    n = w.shape[0] // 2
    half = lambda v, i: None if v is None else v[i * n:(i + 1) * n]
    g, dg = product(q, s, w[:n], sw[:n], half(bias, 0))
    u, du = product(q, s, w[n:], sw[n:], half(bias, 1))
    with np.errstate(over="ignore"):
        a = g / (1 + np.exp(-g))
    # silu' is at most 1.1; exp is good to 2 ulp, then one addition, one division and two products
    return a * u, 1.1 * dg * np.abs(u) + np.abs(a) * du + 8 * E * np.abs(a * u) + 1e-36 * np.abs(u)


def norm(a, da, kind, eps, w, b, w_offset=0.0):
    """(N(a), error bound) from an input with error da.  A row sum in fp32 passes at most 100 roundings on its way (up
    to 64 in a thread, 6 + 16 over the threads); the square root halves the sum's."""
    if kind == "none":
        return a, da
    c, dc = a, da
    if kind == "layer":
        c = a - a.mean(axis=1, keepdims=True)
        dc = da + da.mean(axis=1, keepdims=True) + 100 * E * np.abs(a).mean(axis=1, keepdims=True) + E * np.abs(c)
    sig = np.sqrt((c ** 2).mean(axis=1, keepdims=True) + eps)
    rel = 54 * E + np.sqrt((dc ** 2).mean(axis=1, keepdims=True)) / sig
    k = 1.0 if w is None else w_offset + w
    v = c / sig * k
    dv = np.abs(k) / sig * dc + np.abs(v) * (rel + 4 * E)
    if b is None:
        return v, dv
    return v + b, dv + E * np.abs(v + b)


def block_norm(z, h, post, pre, post_w=None, post_b=None, pre_w=None, pre_b=None, gate=None, gate_rows=1,
               res_scale=1.0, gate_scale=1.0, eps=1e-6, w_offset=0.0):
    """((r, bound), (x, bound))."""
    f = lambda v: np.float64(np.float32(v))  # the constants are fp32
    eps, w_offset, res_scale, gate_scale = f(eps), f(w_offset), f(res_scale), f(gate_scale)
    u, du = norm(z, np.zeros_like(z), post, eps, post_w, post_b, w_offset)
    if gate is not None:
        g = gate[np.arange(z.shape[0]) // gate_rows]
        u, du = u * g, (du + E * np.abs(u)) * np.abs(g)
    u, du = u * gate_scale, (du + E * np.abs(u)) * abs(gate_scale)
    r, dr = u, du
    if h is not None:
        r = res_scale * h + u
        dr = du + E * np.abs(res_scale * h) + E * np.abs(r)
    return (r, dr), norm(r, dr, pre, eps, pre_w, pre_b, w_offset)


def check(got, ref, bound, out):
    """Every value within its bound plus half an ulp of the output type; the same values not finite."""
    got = widen(got) if not isinstance(got, np.ndarray) else got.astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    off = np.abs(got - ref) - bound - half_ulp(ref, out) * (1 + 1e-6)
    worst = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert np.isfinite(got).all()
    assert off.size == 0 or off[worst] <= 0, "at %s: %r, expected %r within %g" % (
        worst, got[worst], ref[worst], bound[worst] if np.ndim(bound) else bound)


def plan(ids, experts):
    """(offsets, rows, pos) by a stable sort."""
    flat = ids.reshape(-1)
    top = ids.shape[1]
    order = [i for e in range(experts) for i in np.flatnonzero(flat == e)]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])]).astype(np.int32)
    pos = np.full(flat.size, -1, np.int32)
    pos[order] = np.arange(len(order))
    return offsets, (np.asarray(order, np.int64) // top).astype(np.int32), pos.reshape(ids.shape)
