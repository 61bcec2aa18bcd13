"""The whole expert layer against its 64-bit form, in every way that it is run: one token in two launches, one token
through the plan, short and long groups, dropped pairs, experts chosen twice.

The bound is derived.  A hidden value is off by q8ref.gated's bound dh, the row's 8-bit scale by the relative dh at its
largest value (and one rounding).  A hidden integer may differ by one where its quotient lies within twice dh (its own
error and the scale's) and a rounding of a tie: one step of it through the output weights.  The output product adds three
roundings, the join one for each slot and one.
"""
import numpy as np
import pytest

import q8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def layer64(q, s, ids, p, w_in, s_in, w_out, s_out):
    """(y, bound) of tokens in 8 bits."""
    y, lim = np.zeros((q.shape[0], w_out.shape[1])), np.zeros((q.shape[0], w_out.shape[1]))
    e_ = q8ref.E
    for ex in range(w_out.shape[0]):
        tok, slot = np.nonzero(ids == ex)
        if tok.size == 0:
            continue
        h, dh = q8ref.gated(q[tok], s[tok], w_in[ex], s_in[ex])
        at = np.abs(h).argmax(axis=1)[:, None]
        big, dbig = np.take_along_axis(np.abs(h), at, 1), np.take_along_axis(dh, at, 1)
        hs = big / 127
        dscale = dbig / big + e_
        v = h / hs
        near = np.abs(np.abs(v - np.floor(v)) - 0.5) * hs <= dh + np.abs(h) * (dscale + e_)
        w, sw = w_out[ex].astype(np.float64), s_out[ex].astype(np.float64)
        z = (np.clip(np.rint(v), -127, 127) @ w.T) * hs * sw       # the integers' sum is exact
        dz = (near.astype(np.float64) @ np.abs(w).T) * hs * sw + np.abs(z) * (dscale + 3 * e_)
        pw = p[tok, slot].astype(np.float64)[:, None]
        np.add.at(y, tok, pw * z)
        np.add.at(lim, tok, pw * dz + (ids.shape[1] + 1) * e_ * np.abs(pw * z))
    return y, lim + 1e-37


@pytest.mark.parametrize("t,e,top,d,i", [
    (1, 4, 2, 512, 1024), (1, 8, 7, 300, 1000), (1, 9, 8, 300, 500), (1, 3, 2, 130, 24100), (2, 8, 2, 1024, 1792),
    (20, 6, 3, 200, 333), (300, 8, 2, 257, 640), (333, 64, 4, 512, 256), (900, 3, 2, 384, 300)])
@pytest.mark.parametrize("how", ["distinct", "dropped", "twice"])
def test_against_64_bits(t, e, top, d, i, how):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    print("experts", t, e, top, d, i, how, flush=True)
    g = np.random.default_rng([t, e, top, d, i])
    ids = np.argsort(g.random((t, e)), axis=1)[:, :top].astype(np.int32)
    if how == "dropped":
        ids[g.random(ids.shape) < 0.3] = -1
    elif how == "twice" and top > 1:
        ids[:, 1] = ids[:, 0]
    p = g.random((t, top)).astype(np.float32)
    w = lambda n, k: np.clip(np.rint(g.standard_normal((e, n, k)) * 32), -127, 127).astype(np.int8)
    sc = lambda n, k: (g.uniform(0.5, 1.5, (e, n)) / (32 * k ** 0.5)).astype(np.float32)
    w_in, s_in, w_out, s_out = w(2 * i, d), sc(2 * i, d), w(d, i), sc(d, i)
    x = g.standard_normal((t, d)).astype(np.float32)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    y = vq.Q8Experts(*map(cu, (w_in, s_in, w_out, s_out)))(cu(x), cu(ids), cu(p))
    q, s = q8ref.quantize(x.astype(np.float64))
    ref, bound = layer64(q, s, ids, p, w_in, s_in, w_out, s_out)
    q8ref.check(y, ref, bound, "f32")
    if how == "distinct":
        assert np.abs(ref).max() > 0.1
