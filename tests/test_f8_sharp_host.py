"""The sharp check of the gated feed-forward layer on the host: what a right layer is off by passes, mistakes do not."""
import numpy as np
import pytest

import f8ref
import f8sharp

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", params=[(40, 512, 2000), (96, 256, 9300)])
def layer(request):
    m, d, i = request.param
    g = np.random.default_rng([m, d, i])
    e4 = lambda *s: f8ref.e4m3(np.clip(g.standard_normal(s) * 100, -448, 448)) * 1e-3
    x, in64, out64 = g.standard_normal((m, d)), e4(2 * i, d) / d ** 0.5, e4(d, i) / i ** 0.5
    return g, x, in64, out64, f8sharp.mlp64(x, in64, out64)


def _off(y, ref, out="bf16"):
    off, limit = f8sharp.beyond_rounding(torch.from_numpy(y).to(f8sharp.DT[out]), ref, out)
    return off / limit


def _from(g, x, in64, out64, spread):
    """The layer with sums of gate and up that are off by `spread` of their own."""
    i = in64.shape[0] // 2
    gate, up = x @ in64[:i].T, x @ in64[i:].T
    gate, up = (v + spread * v.std() * g.standard_normal(v.shape) for v in (gate, up))
    q, s = f8ref.quantize(gate / (1 + np.exp(-gate)) * up)
    return (q * f8ref.spread(s, *q.shape, 1)) @ out64.T


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_sums(layer, out):
    g, x, in64, out64, (y, _) = layer
    assert _off(y, y, out) <= 0.5
    assert _off(_from(g, x, in64, out64, 3e-7), y, out) <= 1   # sums in fp32
    assert _off(_from(g, x, in64, out64, 1.4e-5), y, out) > 1  # sums of the 8-bit matrix instruction


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_mistakes(layer, out):
    g, x, in64, out64, (y, h) = layer
    m, i = h.shape
    block = slice(128, 256)
    less, twice, moved, scale = (h.copy() for _ in range(4))
    less[m // 2, block] = 0                                    # one block of one row is missing
    twice[m // 2, block] *= 2                                  # another block's scale
    moved[:, :-1] = h[:, 1:]                                   # columns shifted by one
    scale[:, block] *= 1.1
    wrong = [np.zeros_like(y), y * 1.1, np.full_like(y, np.nan)] + [v @ out64.T for v in (less, twice, moved, scale)]
    for k, bad in enumerate(wrong):
        assert not _off(bad, y, out) <= 1, k
    swapped = y.copy()
    swapped[[0, 1]] = y[[1, 0]]
    assert _off(swapped, y, out) > 1
