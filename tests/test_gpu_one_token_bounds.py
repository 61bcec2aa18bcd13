"""The bound of the expert layer's two-launch form for one token: its experts' hidden rows in LDS together, 63 KB less
8 KB of sums for each.  On both sides of it the layer gives the bits of its parts called one by one, and the routing plan
at the start of the workspace is written exactly where the form is not taken.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def longest(top):
    """Columns of the hidden rows, whole 128-byte steps."""
    return (63 * 1024 // top - 8192) // 128 * 128


@pytest.mark.parametrize("top", [1, 2, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("over", [0, 1])
def test_both_sides(top, over):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    inner = max(longest(top), 0) + over
    if inner == 0:
        pytest.skip("no row is short enough")
    e, d = top + 1, 130
    g = np.random.default_rng([top, over])
    dev = lambda a: torch.from_numpy(a).cuda()
    w = lambda n, k: vq.q8_pad(dev(g.integers(-127, 128, (e, n, k)).astype(np.int8)))
    s = lambda n: dev(g.uniform(1e-4, 3e-4, (e, n)).astype(np.float32))
    w_in, s_in, w_out, s_out = w(2 * inner, d), s(2 * inner), w(d, inner), s(d)
    x, p = dev(g.standard_normal((1, d)).astype(np.float32)), dev(g.random((1, top)).astype(np.float32))
    ids = dev(g.permutation(e)[:top].astype(np.int32).reshape(1, top))
    ws = torch.full((vq.q8_experts_workspace_bytes(1, top, e, d, inner),), 0xA5, dtype=torch.uint8, device="cuda")
    y = vq.q8_experts(x, ids, p, w_in, s_in, w_out, s_out, inner, ws)
    planned = bool((ws[:4 * (e + 1)] != 0xA5).any())
    assert planned == (longest(top) < inner)

    off, rows, pos = vq.expert_plan(ids, e)
    q, qs = vq.q8_quantize(x)
    h = vq.q8_gemm_grouped(off, rows, q, qs, w_in, s_in, None, d, top, gated=True)
    hq, hs = vq.q8_quantize(h)
    z = vq.q8_gemm_grouped(off, None, hq, hs, w_out, s_out, None, inner, top)
    assert bool(y.any()) and torch.equal(y, vq.expert_combine(z, pos, p))
