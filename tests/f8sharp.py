"""Sharp checks of the gated feed-forward layer in 8-bit floats: how far its outputs are from the 64-bit form beyond their own
rounding, as a root mean square.

A hidden row is cut to e4m3, so an error of g and u shows where it takes a hidden value over the border of two steps.  A value v
whose error is dv is taken over with the probability 2 |dv| / step, and is then off by a step of at most 2^-3 |v|: on average
dv moves it by (2 |dv| 2^-3 |v|)^(1/2) (rms).  Sums in fp32 leave g and u an error of some 3e-7 of their spread, h = silu(g) u
twice that, half of it in the mean, and E|v| is below the spread: (2^-2 * 5e-7)^(1/2) = 3.6e-4 of the hidden rows' norm, and of
the outputs', which are sums of them with weights of no order.  The second product's own sums add 1.4e-5.  Half as much again
is BEYOND.  Sums that are off by 1.4e-5 of their spread come to 0.9e-3 to 1.3e-3."""
from __future__ import annotations

import numpy as np
import torch

import f8ref

BEYOND = 5e-4
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def mlp64(x, in64, out64):
    """(y, hidden values) of the layer: tokens x (values), weights [2 I, D] and [D, I]; the hidden rows are cut from fp32."""
    i = in64.shape[0] // 2
    g, u = x @ in64[:i].T, x @ in64[i:].T
    with np.errstate(over="ignore"):
        q, s = f8ref.quantize(g / (1 + np.exp(-g)) * u)
    h = q * f8ref.spread(s, *q.shape, 1)
    return h @ out64.T, h


def beyond_rounding(got, ref, out):
    """(how far `got` is from `ref`, relative to its norm, beyond what rounding `ref` to the type `out` costs; its limit).
    Infinite where `got` is not finite.  Two sums of n squares of evenly spread rounding errors differ by 1.3 n^(-1/2) of
    themselves (one standard deviation of independent ones); the limit leaves four."""
    got = f8ref.widen(got) if not isinstance(got, np.ndarray) else got.astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    norm = (ref ** 2).sum()
    own = ((torch.from_numpy(ref).to(DT[out]).double().numpy() - ref) ** 2).sum() / norm
    sq = ((got - ref) ** 2).sum() / norm - own
    return (max(sq, 0.0) ** 0.5 if np.isfinite(sq) else np.inf), (BEYOND ** 2 + 4 * 1.3 * ref.size ** -0.5 * own) ** 0.5
