"""GPU parity of the 8-bit products and their quantizer (vq_q8_quantize, vq_q8_gemm, vq_q8_linear, Q8Linear) against
64-bit references.

The integers and scales have to be equal (both are fp32 by definition).  The product's int32 sums are exact, so y is
held to three fp32 roundings of the scaled sum, one for the bias and half an ulp of the output type.
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


def _x(g, m, k, dt, spread=1.0):
    x = g.standard_normal((m, k)) * spread
    x[:, g.random(k) < 0.01] *= 10
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt]).cuda()


def _w(g, n, k):
    w = np.clip(np.rint(g.standard_normal((n, k)) * 40), -127, 127).astype(np.int8)
    return w, g.uniform(0.5, 1.5, n).astype(np.float32) * np.float32(6e-4)


def _q(vq, w):
    return vq.q8_pad(torch.from_numpy(w).cuda())


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (5, 128), (2, 129), (4, 511), (9, 1000), (2, 2048), (3, 4099),
                                 (600, 2056), (2, 8192), (600, 5003), (1, 14336), (2, 28672), (513, 16384), (1, 40001),
                                 (1, 65536)])
def test_quantize(vq, m, k, dt):
    g = np.random.default_rng([m, k])
    x = _x(g, m, k, dt)
    q, s = vq.q8_quantize(x)
    rq, rs = q8ref.quantize(q8ref.widen(x))
    torch.cuda.synchronize()
    assert q.shape == (m, vq.q8_row_bytes(k)) and vq.q8_row_bytes(k) % 128 == 0
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q[:, :k].cpu().numpy(), rq)
    assert not q[:, k:].any()


def test_quantize_special_rows(vq):
    x = torch.randn((12, 300), generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 17] = float("nan")
    x[2, 299] = float("inf")
    x[3, 0] = -float("inf")
    x[4] *= 1e-38          # subnormal and barely normal values: the scale is subnormal
    x[5] = 0
    x[5, 5] = 1e-45        # the scale rounds to zero
    x[6] *= 1e37           # large, finite
    x[7] = 0
    x[7, 1], x[7, 2] = 2.0, 1.0   # a value of half the largest: 63.5 is a tie
    x[8] *= 2e-33
    x[9] = -0.0
    xd = x.cuda()
    q, s = vq.q8_quantize(xd)
    rq, rs = q8ref.quantize(x.numpy().astype(np.float64))
    s = s.cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(rs)) and np.array_equal(s[~np.isnan(rs)], rs[~np.isnan(rs)])
    assert np.array_equal(q[:, :300].cpu().numpy(), rq)


def test_quantize_row_stride_and_alignment(vq):
    g = np.random.default_rng(5)
    big = _x(g, 40, 1111, "bf16")
    view = big[3:36, 5:706]         # odd offset and stride
    q, s = vq.q8_quantize(view)
    q2, s2 = vq.q8_quantize(view.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q3, s3 = vq.q8_quantize(big[::7, 5:706])
    q4, s4 = vq.q8_quantize(big[::7, 5:706].contiguous())
    assert torch.equal(q3, q4) and torch.equal(s3, s4)


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 100, 130), (2, 17, 4096), (1, 4096, 4096), (5, 333, 1000), (16, 64, 14336),
          (17, 100, 256), (33, 65, 640), (37, 203, 4099), (64, 129, 2048), (65, 128, 128), (66, 257, 4096),
          (128, 130, 8192), (130, 1030, 200), (200, 1000, 300), (257, 640, 1152), (300, 4100, 520), (1000, 333, 777),
          (2049, 384, 256), (5, 2, 65536), (70, 3, 65536), (138, 142, 17163), (100, 300, 7168), (60, 1100, 9000),
          (300, 5003, 600), (257, 3000, 1025), (150, 9000, 640), (260, 17000, 257)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out,bias", [("f32", False), ("bf16", True), ("f16", True)])
def test_gemm(vq, m, n, k, out, bias):
    print("q8_gemm", m, n, k, out, flush=True)
    g = np.random.default_rng([m, n, k])
    x = _x(g, m, k, "f32")
    w, sw = _w(g, n, k)
    b = (g.standard_normal(n) * 0.3).astype(np.float16) if bias else None
    q, s = vq.q8_quantize(x)
    args = (q, s, _q(vq, w), torch.from_numpy(sw).cuda(), torch.from_numpy(b).cuda() if bias else None, k)
    nb = vq.q8_gemm_workspace_bytes(m, n, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
    y = vq.q8_gemm(*args, ws=ws, y_dtype=DT[out])
    ref, bound = q8ref.product(q[:, :k].cpu().numpy(), s.cpu().numpy(), w, sw, b)
    q8ref.check(y, ref, bound, out)
    # without a workspace the same bits, and from x in one call too
    assert torch.equal(y, vq.q8_gemm(*args, y_dtype=DT[out]))
    lw = torch.empty(vq.q8_linear_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    assert torch.equal(y, vq.q8_linear(x, *args[2:5], lw, y_dtype=DT[out]))


@pytest.mark.parametrize("m,n,k", [(4200, 4100, 130), (5000, 4999, 100)])
def test_gemm_many_tiles(vq, m, n, k):
    """Enough 256 x 256 tiles to fill the CUs: 289 of them (33 in the second round, cut in halves) and 400."""
    g = np.random.default_rng([m, n, k])
    x = _x(g, m, k, "bf16")
    w, sw = _w(g, n, k)
    q, s = vq.q8_quantize(x)
    y = vq.q8_gemm(q, s, _q(vq, w), torch.from_numpy(sw).cuda(), None, k, y_dtype=torch.float32)
    ref, bound = q8ref.product(q[:, :k].cpu().numpy(), s.cpu().numpy(), w, sw)
    q8ref.check(y, ref, bound, "f32")


@pytest.mark.parametrize("n,k", [(1, 1), (70, 57345), (3, 60000), (5000, 129), (13000, 333), (256, 14336)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_one_token(vq, n, k, dt):
    """The form that cuts its token inside the product, and rows too long for it: the same bits as the two steps."""
    g = np.random.default_rng([n, k])
    x = _x(g, 1, k, dt)
    w, sw = _w(g, n, k)
    b = (g.standard_normal(n) * 0.3).astype(np.float16)
    wd, swd, bd = _q(vq, w), torch.from_numpy(sw).cuda(), torch.from_numpy(b).cuda()
    ws = torch.empty(vq.q8_linear_workspace_bytes(1, n, k), dtype=torch.uint8, device="cuda")
    y = vq.q8_linear(x, wd, swd, bd, ws, y_dtype=torch.float32)
    q, s = q8ref.quantize(q8ref.widen(x))
    ref, bound = q8ref.product(q, s, w, sw, b)
    q8ref.check(y, ref, bound, "f32")
    q2, s2 = vq.q8_quantize(x)
    assert torch.equal(y, vq.q8_gemm(q2, s2, wd, swd, bd, k, y_dtype=torch.float32))
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[0, k // 2] = bad
        assert bool(torch.isnan(vq.q8_linear(x2, wd, swd, bd, ws)).all())
    zero = vq.q8_linear(torch.zeros_like(x), wd, swd, bd, ws, y_dtype=torch.float32)
    assert torch.equal(zero[0], bd.float())


def test_gemm_extreme_integers(vq):
    """All products at their largest: K = 65536 sums of 127 * -128 stay exact."""
    for m in (1, 16, 80):
        q = torch.full((m, 65536), 127, dtype=torch.int8, device="cuda")
        w = torch.full((130, 65536), -128, dtype=torch.int8, device="cuda")
        one = lambda n: torch.ones(n, device="cuda")
        y = vq.q8_gemm(q, one(m), w, one(130), None, 65536, y_dtype=torch.float32)
        assert bool((y == float(np.float32(-127 * 128 * 65536))).all())


@pytest.mark.parametrize("m", [3, 100])
def test_nan_rows_stay_apart(vq, m):
    g = np.random.default_rng(m)
    x = _x(g, m, 500, "f16")
    w, sw = _w(g, 70, 500)
    lay = vq.Q8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(sw).cuda())
    clean = lay(x)
    x2 = x.clone()
    x2[1, 77] = float("inf")
    y = lay(x2)
    assert bool(torch.isnan(y[1]).all())
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("m", [2, 70])
def test_offsets_past_32_bits(vq, m):
    """4.4 GB of weights: the last rows lie past 2^32 bytes."""
    n, k = 270001, 16384
    gen = torch.Generator(device="cuda").manual_seed(m)
    w = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    sw = torch.rand((n,), generator=gen, device="cuda")
    x = torch.randn((m, k), generator=gen, device="cuda").half()
    q, s = vq.q8_quantize(x)
    y = vq.q8_gemm(q, s, w, sw, None, k, y_dtype=torch.float32)
    rows = [0, 131071, 131072, 262143, 262144, n - 129, n - 17, n - 1]
    ref, bound = q8ref.product(q.cpu().numpy(), s.cpu().numpy(), w[rows].cpu().numpy(), sw[rows].cpu().numpy())
    q8ref.check(y[:, rows], ref, bound, "f32")


def test_linear_layer(vq):
    g = np.random.default_rng(9)
    w = torch.from_numpy((g.standard_normal((200, 333)) * 0.02).astype(np.float32)).cuda()
    b = torch.from_numpy(g.standard_normal(200).astype(np.float16)).cuda()
    lay = vq.Q8Linear.from_weight(w, b)
    x = _x(g, 12, 333, "bf16").reshape(3, 4, 333)
    y = lay(x)
    assert y.shape == (3, 4, 200) and y.dtype == torch.bfloat16
    q, s = q8ref.quantize(q8ref.widen(x.reshape(12, 333)))
    wq, sw = q8ref.quantize(q8ref.widen(w))
    ref, bound = q8ref.product(q, s, wq, sw, b.cpu().numpy())
    q8ref.check(y.reshape(12, 200), ref, bound, "bf16")
    q2, s2 = vq.q8_quantize(x.reshape(12, 333))
    assert torch.equal(lay.forward_q8(q2, s2).reshape(3, 4, 200), y)
    assert torch.equal(lay(x.transpose(0, 1)), y.transpose(0, 1))     # an input that is not contiguous
    assert lay(x[:0]).shape == (0, 4, 200)
    # 8-bit weights keep the layer close to the dense one: half a step of each of 333 weights and of each activation
    dense = q8ref.widen(x.reshape(12, 333)) @ q8ref.widen(w).T + q8ref.widen(b)
    lim = 0.5 * (np.abs(q8ref.widen(x.reshape(12, 333))).sum(1)[:, None] * sw[None, :].astype(np.float64)
                 + s[:, None].astype(np.float64) * np.abs(q8ref.widen(w)).sum(1)[None, :]) * 1.01
    assert (np.abs(q8ref.widen(y.reshape(12, 200)) - dense) <= lim + q8ref.half_ulp(dense, "bf16")).all()


def test_other_stream_and_graph(vq):
    g = np.random.default_rng(11)
    w, sw = _w(g, 300, 700)
    lay = vq.Q8Linear(torch.from_numpy(w).cuda(), torch.from_numpy(sw).cuda())
    for m in (2, 90):
        x = _x(g, m, 700, "f16")
        want = lay(x)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got = lay(x)
        st.synchronize()
        assert torch.equal(got, want)
        buf = x.clone()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st):
            lay(buf)
        st.synchronize()
        with torch.cuda.graph(gr, stream=st):
            out = lay(buf)
        for k in range(3):
            x2 = _x(np.random.default_rng(k), m, 700, "f16")
            buf.copy_(x2)
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, lay(x2)), k


def test_refusals(vq):
    x = torch.zeros((4, 100), device="cuda", dtype=torch.float16)
    w = vq.q8_pad(torch.zeros((8, 100), device="cuda", dtype=torch.int8))
    sw = torch.ones(8, device="cuda")
    ws = torch.empty(vq.q8_linear_workspace_bytes(4, 8, 100), dtype=torch.uint8, device="cuda")
    q, s = vq.q8_quantize(x)
    with pytest.raises(ValueError):
        vq.q8_quantize(x.t())
    with pytest.raises(ValueError):
        vq.q8_quantize(x[0])
    with pytest.raises(ValueError):
        vq.q8_quantize(x[:1].expand(4, 100))
    with pytest.raises(TypeError):
        vq.q8_quantize(x.int())
    with pytest.raises(ValueError):
        vq.q8_quantize(x.cpu())
    with pytest.raises(TypeError):
        vq.q8_pad(x)
    with pytest.raises(ValueError):
        vq.q8_gemm(q, s, w, sw, None, 200)
    with pytest.raises(ValueError):
        vq.q8_gemm(q, s[:3], w, sw, None, 100)
    with pytest.raises(ValueError):
        vq.q8_linear(x, w, sw[:7], None, ws)
    with pytest.raises(TypeError):
        vq.q8_linear(x, w, sw.half(), None, ws)
    with pytest.raises(ValueError):
        vq.q8_linear(x, w, sw, None, ws, out=torch.empty((4, 9), device="cuda"))
    for bad in (None, ws[:64]):
        with pytest.raises(vq.VQError):
            vq.q8_linear(x, w, sw, None, bad)
    with pytest.raises(vq.VQError) as e:
        vq.q8_quantize(torch.zeros((1, 65537), device="cuda"))
    assert e.value.status == vq.VQ_ERR_SHAPE
