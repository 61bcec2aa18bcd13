"""GPU parity of vq_block_norm against a 64-bit reference whose error bound follows the fp32 roundings of each step
(q8ref.block_norm), over types, lengths, strides, norm kinds and gates; the 8-bit output equals the quantizer's on the
same fp32 values, bit for bit.
"""
import numpy as np
import pytest

import q8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as g

    g.lib()
    return g


def _t(g, shape, dt, spread=1.0, shift=0.0):
    return torch.from_numpy((g.standard_normal(shape) * spread + shift).astype(np.float32)).to(DT[dt]).cuda()


def _inputs(g, m, d, zt, ht, wt, post, pre, bias, gate, gate_rows):
    kw = {"post": post, "pre": pre, "gate_rows": gate_rows}
    if post != "none":
        kw["post_weight"] = _t(g, d, wt, 0.1, 0.5)
        kw["post_bias"] = _t(g, d, wt, 0.1) if bias else None
    if pre != "none":
        kw["pre_weight"] = _t(g, d, wt, 0.1, 1.0)
        kw["pre_bias"] = _t(g, d, wt, 0.1) if bias else None
    if gate == "channel":
        kw["gate"] = _t(g, d, zt)
    elif gate == "rows":
        kw["gate"] = _t(g, (-(-m // gate_rows), d), zt)
    return _t(g, (m, d), zt, 0.7, 0.2), None if ht is None else _t(g, (m, d), ht, 2.0), kw


def _ref(z, h, kw):
    w = lambda k: None if kw.get(k) is None else q8ref.widen(kw[k])
    gate, rows = w("gate"), kw["gate_rows"]
    if gate is not None and gate.ndim == 1:
        gate, rows = gate[None], z.shape[0]
    return q8ref.block_norm(q8ref.widen(z), None if h is None else q8ref.widen(h), kw["post"], kw["pre"],
                            w("post_weight"), w("post_bias"), w("pre_weight"), w("pre_bias"), gate, rows,
                            kw.get("res_scale", 1.0), kw.get("gate_scale", 1.0), kw.get("eps", 1e-6),
                            kw.get("weight_offset", 0.0))


@pytest.mark.parametrize("m,d", [(1, 1), (1, 4096), (3, 2), (5, 63), (9, 512), (6, 513), (700, 1000), (33, 1025),
                                 (3, 2049), (520, 2048), (600, 4097), (4, 5003), (515, 8192), (2, 8192), (3, 9000),
                                 (514, 12000), (2, 16384), (2, 20001), (1, 33000), (1, 65536)])
@pytest.mark.parametrize("post,pre,zt,ht,wt,bias,gate,rows", [
    ("none", "rms", "f16", "f16", "f32", False, "none", 1),
    ("rms", "rms", "bf16", "bf16", "bf16", False, "channel", 1),
    ("layer", "layer", "f16", "f32", "f32", True, "rows", 2),
    ("rms", "layer", "f32", "f32", "f16", True, "rows", 1),
    ("layer", "none", "bf16", "f32", "f32", False, "none", 1),
    ("none", "none", "f32", "f16", "f32", False, "channel", 1),
])
def test_block_norm(vq, m, d, post, pre, zt, ht, wt, bias, gate, rows):
    g = np.random.default_rng([m, d])
    z, h, kw = _inputs(g, m, d, zt, ht, wt, post, pre, bias, gate, rows)
    kw |= {"res_scale": 0.9, "gate_scale": 1.3, "eps": 1e-5}
    (r64, dr), (x64, dx) = _ref(z, h, kw)
    r, x = vq.block_norm(z, h, **kw)
    assert r.dtype == h.dtype and x.dtype == z.dtype
    q8ref.check(r, r64, dr, ht)
    q8ref.check(x, x64, dx, zt)
    r2, xf = vq.block_norm(z, h, x_dtype=torch.float32, **kw)
    r3, q, s = vq.block_norm(z, h, q8=True, **kw)
    q2, s2 = vq.q8_quantize(xf)
    assert torch.equal(r2, r) and torch.equal(r3, r) and torch.equal(q, q2) and torch.equal(s, s2)


def test_without_a_residual(vq):
    g = np.random.default_rng(2)
    for gs in (1.0, 0.25):
        z, _, kw = _inputs(g, 7, 300, "bf16", None, "f32", "rms", "rms", False, "none", 1)
        kw["gate_scale"] = gs
        (r64, dr), (x64, dx) = _ref(z, None, kw)
        r, x = vq.block_norm(z, None, **kw)
        q8ref.check(r, r64, dr, "bf16")
        q8ref.check(x, x64, dx, "bf16")
        none, x2 = vq.block_norm(z, None, keep_r=False, **kw)
        assert none is None and torch.equal(x, x2)


def test_weight_offset_in_place_and_strides(vq):
    g = np.random.default_rng(4)
    m, d = 37, 1111
    big = _t(g, (2 * m, d + 9), "f16")
    z = big[::2, 3:3 + d]
    hb = _t(g, (m, d + 5), "f32", 2.0)
    h = hb[:, 1:1 + d]
    w = _t(g, d, "f16", 0.1)
    kw = {"post": "rms", "pre": "rms", "post_weight": w, "pre_weight": w, "weight_offset": 1.0, "gate_rows": 1}
    (r64, dr), (x64, dx) = _ref(z, h, kw)
    r, x = vq.block_norm(z, h, **kw)
    q8ref.check(r, r64, dr, "f32")
    q8ref.check(x, x64, dx, "f16")
    hc = h.contiguous()
    r2, x2 = vq.block_norm(z, hc, r_out=hc, **kw)
    assert r2.data_ptr() == hc.data_ptr() and torch.equal(r2, r) and torch.equal(x2, x)


def test_constant_zero_and_non_finite_rows(vq):
    x = torch.zeros((6, 640), device="cuda")
    x[1] = 3.0                       # no spread: the centred norm gives zeros
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = torch.randn(640, generator=torch.Generator().manual_seed(1))
    for pre in ("rms", "layer"):
        _, y = vq.block_norm(x, pre=pre, eps=1e-5)
        assert not y[0].any() and bool(torch.isnan(y[2]).all())
        assert bool(torch.isfinite(y[4]).all())
        if pre == "layer":
            assert not y[1].any() and bool(torch.isnan(y[3]).all())
        _, q, s = vq.block_norm(x, pre=pre, eps=1e-5, q8=True)
        assert not q[0].any() and float(s[0]) == 0 and bool(torch.isnan(s[2])) and not q[2].any()
        assert bool(torch.isnan(s[3]))
    assert vq.block_norm(x[:0])[1].shape == (0, 640)


def test_then_product(vq):
    """The block's entry as it is used: norms and residual add, then a product on the 8-bit tokens."""
    g = np.random.default_rng(12)
    z, h, kw = _inputs(g, 37, 403, "bf16", "bf16", "f32", "rms", "rms", False, "none", 1)
    w = torch.from_numpy((g.standard_normal((210, 403)) * 0.02).astype(np.float32)).cuda()
    lay = vq.Q8Linear.from_weight(w)
    r, q, s = vq.block_norm(z, h, q8=True, **kw)
    y = lay.forward_q8(q, s, y_dtype=torch.float32)
    ref, bound = q8ref.product(q[:, :403].cpu().numpy(), s.cpu().numpy(), lay.w[:, :403].cpu().numpy(),
                               lay.scale.cpu().numpy())
    q8ref.check(y, ref, bound, "f32")


def test_refusals(vq):
    z = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        vq.block_norm(z, pre="batch")
    with pytest.raises(ValueError):
        vq.block_norm(z, pre_weight=w[:63])
    with pytest.raises(TypeError):
        vq.block_norm(z, post="rms", post_weight=w.half(), pre_weight=w)
    with pytest.raises(ValueError):
        vq.block_norm(z, torch.zeros((4, 65), device="cuda"))
    with pytest.raises(ValueError):
        vq.block_norm(z, gate=torch.ones((3, 64), device="cuda"), gate_rows=2)
    with pytest.raises(ValueError):
        vq.block_norm(z, gate=torch.ones((4, 64), device="cuda"), gate_rows=0)
    with pytest.raises(vq.VQError):
        vq.block_norm(z, pre="none", pre_weight=w)
    with pytest.raises(vq.VQError):
        vq.block_norm(torch.zeros((1, 65537), device="cuda"))
    with pytest.raises(TypeError):
        vq.block_norm(z, z, r_out=torch.zeros((4, 64), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        vq.block_norm(z.cpu())
