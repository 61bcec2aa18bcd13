"""block_norm over any leading dimensions, as the layers that read its output take them: the bits of the same rows in 2-d."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as g

    return g


def _t(seed, *s):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("shape", [(3, 4, 65), (2, 1, 3, 130), (77,), (0, 4, 64), (1, 1, 8)])
@pytest.mark.parametrize("gate", ["none", "channel", "rows"])
def test_batches(vq, shape, gate):
    d = shape[-1]
    z, h = _t(1, *shape).half(), _t(2, *shape)
    m = z.numel() // d
    kw = {"pre": "layer", "post": "rms", "pre_weight": _t(3, d), "pre_bias": _t(4, d), "post_weight": _t(5, d),
          "gate_scale": 0.7}
    if gate == "channel":
        kw["gate"] = _t(6, d)
    elif gate == "rows":
        kw |= {"gate": _t(6, -(-m // 2), d), "gate_rows": 2}
    r2, x2 = vq.block_norm(z.reshape(m, d), h.reshape(m, d), **kw)
    r, x = vq.block_norm(z, h, **kw)
    assert r.shape == x.shape == z.shape and r.dtype == h.dtype and x.dtype == z.dtype
    assert torch.equal(r.reshape(m, d), r2) and torch.equal(x.reshape(m, d), x2)
    r3, q, s = vq.block_norm(z, h, q8=True, **kw)
    rq, q2, s2 = vq.block_norm(z.reshape(m, d), h.reshape(m, d), q8=True, **kw)
    assert torch.equal(r3, r) and torch.equal(q, q2) and torch.equal(s, s2) and q.shape[0] == m
    none, x4 = vq.block_norm(z, h, keep_r=False, **kw)
    assert none is None and torch.equal(x4, x)
    into = h.clone()
    r5, x5 = vq.block_norm(z, into, r_out=into, **kw)       # in place
    assert r5 is into and torch.equal(into, r) and torch.equal(x5, x)


def test_not_contiguous(vq):
    z, h = _t(1, 5, 64, 3).transpose(1, 2), _t(2, 3, 5, 64).transpose(0, 1)
    r, x = vq.block_norm(z, h, pre="rms")
    r2, x2 = vq.block_norm(z.contiguous().reshape(15, 64), h.contiguous().reshape(15, 64), pre="rms")
    assert torch.equal(r.reshape(15, 64), r2) and torch.equal(x.reshape(15, 64), x2)
    e = _t(3, 1, 1, 64).expand(2, 3, 64)
    assert torch.equal(vq.block_norm(e, e)[1], vq.block_norm(e.contiguous(), e.contiguous())[1])


def test_refusals(vq):
    z = _t(1, 2, 3, 64)
    with pytest.raises(ValueError):
        vq.block_norm(z, _t(2, 6, 64))
    with pytest.raises(ValueError):
        vq.block_norm(z, r_out=torch.empty((6, 64), device="cuda"))
    with pytest.raises(ValueError):
        vq.block_norm(z, r_out=torch.empty((3, 2, 64), device="cuda").transpose(0, 1))
    with pytest.raises(TypeError):
        vq.block_norm(z, r_out=torch.empty((2, 3, 64), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        vq.block_norm(z, pre_weight=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        vq.block_norm(z.cpu())
    with pytest.raises(ValueError):
        vq.block_norm(z[0, 0, 0])
