"""The gated feed-forward layer's outputs are off by their own rounding and what fp32 sums take with them, in every type and
way: 16-bit outputs too, whose bound in test_gpu_f8 is wide."""
import numpy as np
import pytest

import f8ref
import f8sharp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = f8sharp.DT


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as g

    g.lib()
    return g


def _weights(vq, g, n, k, halves=1):
    v = f8ref.e4m3(np.clip(g.standard_normal((halves * n, k)) * 100, -448, 448))
    s = g.uniform(0.5, 1.5, (halves * f8ref.blocks(n), f8ref.blocks(k))).astype(np.float32) * np.float32(0.01 / k ** 0.5)
    full = np.concatenate([f8ref.spread(p, n, k, 128) for p in np.split(s, halves)])
    w = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn)
    return w.cuda(), torch.from_numpy(s).cuda(), v * full


# one token, streamed; tiles of every size; hidden rows that the product writes in 8 bits (from some thousand columns and a few
# hundred tokens on), with short tiles and blocks at the ends of both
@pytest.mark.parametrize("m,d,i", [(1, 512, 9000), (5, 1024, 2048), (40, 512, 2000), (77, 640, 5001), (130, 300, 4096),
                                   (513, 256, 9300), (700, 264, 10001), (2049, 384, 6001)])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_beyond_rounding(vq, m, d, i, out):
    g = np.random.default_rng([m, d, i])
    x = torch.from_numpy(g.standard_normal((m, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    w_in, s_in, in64 = _weights(vq, g, i, d, halves=2)
    w_out, s_out, out64 = _weights(vq, g, d, i)
    rows = np.unique(np.concatenate([np.arange(min(m, 24)), np.arange(max(m - 24, 0), m), g.integers(0, m, 48)]))
    q, s = f8ref.quantize(f8ref.widen(x)[rows])
    ref, _ = f8sharp.mlp64(q * f8ref.spread(s, *q.shape, 1), in64, out64)
    print("mlp", m, d, i, out, flush=True)
    y = vq.F8MLP(w_in, s_in, w_out, s_out)(x, DT[out])
    torch.cuda.synchronize()
    off, limit = f8sharp.beyond_rounding(y[torch.from_numpy(rows).cuda()], ref, out)
    print("beyond rounding %.2e of %.2e" % (off, limit), flush=True)
    assert off <= limit
