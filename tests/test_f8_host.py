"""The 8-bit float layers' C entry points and their binding on the host (no GPU): sizes, and every refusal, which has to come
back before anything is launched.  Pointers are made-up aligned addresses: nothing may be read through them."""
import ctypes

import numpy as np
import pytest

import f8ref

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def vq():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    g.lib()
    return g


P = 1 << 20
F16, F32, BAD = 0, 2, 7


def _size(f, *a):
    n = ctypes.c_size_t(12345)
    return f(*a, ctypes.byref(n)), n.value


def test_reference_against_torch():
    """The reference's rounding and decoding are torch's e4m3."""
    q = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy()
    got = f8ref.decode(q)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    v = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s for s in (1e-3, 1e-2, 1, 100)])
    v = np.concatenate([v, got[~np.isnan(got)], (np.arange(-448, 449) / 16.0)]).clip(-448, 448).astype(np.float32)
    assert np.array_equal(f8ref.e4m3(v.astype(np.float64)), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_workspace_sizes(vq):
    lib = vq.lib()
    pad = lambda b: (b + 255) // 256 * 256
    for f in (lib.vq_f8_gemm_workspace_bytes, lib.vq_f8_linear_workspace_bytes):
        for bad in ((-1, 1, 1, 0), (1, -1, 1, 0), (1, 1, 0, 0), (1, 1, 65537, 0), (1, 1 << 30, 1, 1)):
            assert _size(f, *bad)[0] == vq.VQ_ERR_SHAPE
        assert _size(f, 1, 1, 1, 2)[0] == vq.VQ_ERR_UNSUPPORTED
        assert f(64, 128, 256, 0, None) == vq.VQ_ERR_NULL
        for zero in ((0, 128, 256, 0), (64, 0, 256, 1)):
            assert _size(f, *zero) == (0, 0)
    for m, n, k in ((37, 5003, 4099), (128, 8192, 28672), (4096, 14336, 4096)):
        st, part = _size(lib.vq_f8_gemm_workspace_bytes, m, n, k, 0)
        assert st == 0 and part % (4 * m * n) == 0
        assert _size(lib.vq_f8_linear_workspace_bytes, m, n, k, 0) == (
            0, pad(m * vq.q8_row_bytes(k)) + pad(4 * m * vq.f8_blocks(k)) + pad(part))
    assert _size(lib.vq_f8_linear_workspace_bytes, 1, 4096, 4096, 0) == (0, 0)
    f = lib.vq_f8_mlp_workspace_bytes
    assert _size(f, 0, 64, 64) == (0, 0)
    assert _size(f, 3, 512, 300)[1] >= 3 * 300 * 4
    for bad in ((-1, 64, 64), (1, 0, 64), (1, 64, 65537)):
        assert _size(f, *bad)[0] == vq.VQ_ERR_SHAPE
    assert f(1, 1, 1, None) == vq.VQ_ERR_NULL


def test_quantize_refusals(vq):
    f = vq.lib().vq_f8_quantize
    call = lambda rows=4, k=64, br=1, x=P, dt=F16, ld=64, q=P, s=P: f(rows, k, br, x, dt, ld, q, s, None)
    for kw in (dict(rows=-1), dict(k=0), dict(k=65537, ld=65537), dict(ld=63), dict(rows=2 ** 31 - 1, br=128)):
        assert call(**kw) == vq.VQ_ERR_SHAPE, kw
    for kw in (dict(dt=BAD), dict(br=0), dict(br=64), dict(br=-1)):
        assert call(**kw) == vq.VQ_ERR_UNSUPPORTED, kw
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert call(**kw) == vq.VQ_ERR_NULL, kw
    for kw in (dict(x=P + 1), dict(x=P + 2, dt=F32), dict(q=P + 8), dict(s=P + 2)):
        assert call(**kw) == vq.VQ_ERR_ALIGN, kw
    assert call(rows=0, x=None, q=None, s=None) == vq.VQ_OK


def test_product_refusals(vq):
    f = vq.lib().vq_f8_gemm

    def call(m=64, n=64, k=64, q=P, s=P, w=P, sw=P, b=None, g=0, y=P, dt=F16, ws=None, nb=0):
        return f(m, n, k, q, s, w, sw, b, g, y, dt, ws, nb, None)

    for kw in (dict(m=-1), dict(n=-1), dict(k=0), dict(k=65537), dict(n=1 << 30, g=1), dict(m=2 ** 31 - 1, n=2 ** 31 - 1),
               dict(n=2 ** 31 - 1), dict(m=2 ** 31 - 1)):
        assert call(**kw) == vq.VQ_ERR_SHAPE, kw
    for kw in (dict(dt=BAD), dict(g=2), dict(g=-1)):
        assert call(**kw) == vq.VQ_ERR_UNSUPPORTED, kw
    for what in ("q", "s", "w", "sw", "y"):
        assert call(**{what: None}) == vq.VQ_ERR_NULL, what
    for kw in (dict(q=P + 8), dict(w=P + 8), dict(s=P + 2), dict(sw=P + 2), dict(b=P + 1), dict(y=P + 1),
               dict(y=P + 2, dt=F32)):
        assert call(**kw) == vq.VQ_ERR_ALIGN, kw
    need = vq.f8_gemm_workspace_bytes(128, 8192, 28672)
    assert need > 0
    assert call(128, 8192, 28672, ws=P, nb=255) == vq.VQ_ERR_BUFFER_SIZE
    assert call(128, 8192, 28672, ws=P + 128, nb=need) == vq.VQ_ERR_ALIGN
    for kw in (dict(m=0), dict(n=0)):
        assert call(q=None, s=None, w=None, sw=None, y=None, **kw) == vq.VQ_OK


def test_linear_refusals(vq):
    f = vq.lib().vq_f8_linear

    def call(m=64, n=64, k=64, x=P, dx=F16, ld=None, w=P, sw=P, b=None, g=0, y=P, dy=F16, ws=P, nb=1 << 40):
        return f(m, n, k, x, dx, k if ld is None else ld, w, sw, b, g, y, dy, ws, nb, None)

    for kw in (dict(m=-1), dict(n=-1), dict(k=0), dict(k=65537), dict(ld=63), dict(m=2 ** 31 - 1, n=2 ** 31 - 1)):
        assert call(**kw) == vq.VQ_ERR_SHAPE, kw
    for kw in (dict(dx=BAD), dict(dy=BAD), dict(g=2)):
        assert call(**kw) == vq.VQ_ERR_UNSUPPORTED, kw
    for kw in (dict(x=None), dict(w=None), dict(sw=None), dict(y=None), dict(ws=None)):
        assert call(**kw) == vq.VQ_ERR_NULL, kw
    for kw in (dict(x=P + 1), dict(w=P + 8), dict(sw=P + 2), dict(b=P + 1), dict(y=P + 1), dict(ws=P + 128)):
        assert call(**kw) == vq.VQ_ERR_ALIGN, kw
    need = vq.f8_linear_workspace_bytes(64, 64, 64)
    assert call(nb=need - 1) == vq.VQ_ERR_BUFFER_SIZE
    assert call(m=0, x=None, w=None, sw=None, y=None, ws=None) == vq.VQ_OK


def test_mlp_refusals(vq):
    f = vq.lib().vq_f8_mlp

    def call(m=64, d=64, i=128, x=P, dx=F16, ld=None, wi=P, si=P, wo=P, so=P, y=P, dy=F16, ws=P, nb=1 << 62):
        return f(m, d, i, x, dx, d if ld is None else ld, wi, si, wo, so, y, dy, ws, nb, None)

    for kw in (dict(m=-1), dict(d=0), dict(i=0), dict(i=65537), dict(ld=63), dict(m=2 ** 31 - 1, d=65536, i=65536)):
        assert call(**kw) == vq.VQ_ERR_SHAPE, kw
    for kw in (dict(dx=BAD), dict(dy=BAD)):
        assert call(**kw) == vq.VQ_ERR_UNSUPPORTED, kw
    for what in ("x", "wi", "si", "wo", "so", "y", "ws"):
        assert call(**{what: None}) == vq.VQ_ERR_NULL, what
    for kw in (dict(x=P + 1), dict(wi=P + 8), dict(wo=P + 8), dict(si=P + 2), dict(so=P + 2), dict(y=P + 1),
               dict(ws=P + 128)):
        assert call(**kw) == vq.VQ_ERR_ALIGN, kw
    assert call(nb=vq.f8_mlp_workspace_bytes(64, 64, 128) - 1) == vq.VQ_ERR_BUFFER_SIZE
    assert call(m=0, x=None, wi=None, si=None, wo=None, so=None, y=None, ws=None) == vq.VQ_OK


def test_binding_refusals(vq):
    e4m3 = torch.float8_e4m3fn
    w = torch.zeros((4, 128), dtype=e4m3)
    with pytest.raises(TypeError):
        vq.f8_pad(torch.zeros((4, 100), dtype=torch.int8))
    p = vq.f8_pad(torch.ones((4, 100)).to(e4m3))
    assert p.shape == (4, 128) and p.dtype == e4m3 and not p[:, 100:].float().any() and bool((p[:, :100].float() == 1).all())
    for call in (lambda: vq.f8_quantize(torch.zeros((2, 8))), lambda: vq.F8Linear(w, torch.zeros((1, 1))),
                 lambda: vq.f8_gemm(w, torch.zeros((1, 4)), w, torch.zeros((1, 1)), None, 128)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="even number of rows"):
        vq.f8.f8_linear.__globals__["_outputs"](torch.zeros((3, 8)), True)


def test_layer_refuses_another_width(vq):
    """Columns that the padding of rows hides: w_in for 100 columns beside w_out for 120."""
    e4 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match=r"w_in must be \[32, 120\]"):
        vq.F8MLP(e4(32, 100), torch.zeros((2, 1)), e4(120, 16), torch.zeros((1, 1)))


@pytest.mark.parametrize("gate,up,out", [((16, 100), (16, 100), (120, 16)),   # columns that the padding of rows hides
                                         ((16, 128), (16, 128), (100, 16)),   # columns that would be cut off
                                         ((17, 100), (15, 100), (100, 16)),   # rows that add up to both halves
                                         ((16, 100), (16, 99), (100, 16)), ((32, 100), (0, 100), (100, 16)),
                                         ((16, 100), (16, 100), (100, 17))])
def test_from_weights_refuses_other_shapes(vq, monkeypatch, gate, up, out):
    cut = []
    monkeypatch.setattr(vq.f8, "f8_quantize", lambda w, *a: cut.append(w) or (
        torch.zeros((w.shape[0], vq.q8_row_bytes(w.shape[1])), dtype=torch.float8_e4m3fn),
        torch.zeros((vq.f8_blocks(w.shape[0]), vq.f8_blocks(w.shape[1])))))
    monkeypatch.setattr(vq.q8, "_device", lambda t, what: -1)
    with pytest.raises(ValueError, match="gate and up must be"):
        vq.F8MLP.from_weights(*(torch.zeros(s) for s in (gate, up, out)))
    assert not cut
    layer = vq.F8MLP.from_weights(*(torch.zeros(s) for s in ((16, 100), (16, 100), (100, 16))))
    assert (layer.features, layer.inner) == (100, 16) and len(cut) == 3


def test_outputs_over_the_input_are_refused(vq):
    """Tokens that are cut inside the product are read by every workgroup, while others store: y may not be x."""
    f, out = vq.lib().vq_f8_linear, 1 << 21
    for m in (1, 8, 64):  # the tokens cut inside, and by a launch in front
        assert f(m, 64, 64, P, F16, 64, out, out, None, 0, P, F16, out, 1 << 40, None) == vq.VQ_ERR_UNSUPPORTED
