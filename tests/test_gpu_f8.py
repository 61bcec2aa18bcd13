"""GPU parity of the 8-bit float layers (vq_f8_*, F8Linear, F8MLP) against 64-bit references.

Values and scales of the cutting have to be equal (both are fp32 by definition).  Products of small whole numbers with
scales that are powers of two are exact in every order and have to be equal bit for bit; others are held to the bound of
f8ref.product and half an ulp of the output type.
"""
import numpy as np
import pytest

import f8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4 = torch.float8_e4m3fn


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


def _w(vq, g, n, k, halves=1):
    """(padded weights, scales, their values): e4m3 with a scale for each block, a set of blocks for each of `halves`."""
    v = f8ref.e4m3(np.clip(g.standard_normal((halves * n, k)) * 100, -448, 448))
    s = g.uniform(0.5, 1.5, (halves * f8ref.blocks(n), f8ref.blocks(k))).astype(np.float32) * np.float32(2e-4)
    w = vq.f8_pad(torch.from_numpy(v.astype(np.float32)).to(E4)).cuda()
    full = np.concatenate([f8ref.spread(p, n, k, 128) for p in np.split(s, halves)])
    return w, torch.from_numpy(s).cuda(), v * full


def _tokens(x):
    """The values of tokens cut to 8 bits."""
    x = f8ref.widen(x)
    q, s = f8ref.quantize(x)
    return q * f8ref.spread(s, *x.shape, 1)


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (5, 128), (2, 129), (17, 511), (40, 1000), (9, 2048), (3, 4099), (600, 136),
                                 (1, 65536)])
def test_quantize(vq, m, k, dt):
    x = _x(np.random.default_rng([m, k]), m, k, dt)
    for rows in (1, 128):
        q, s = vq.f8_quantize(x, rows)
        rq, rs = f8ref.quantize(f8ref.widen(x), rows)
        torch.cuda.synchronize()
        assert q.shape == (m, vq.q8_row_bytes(k)) and q.dtype == E4
        want = rs.T if rows == 1 else rs
        assert np.array_equal(s.cpu().numpy().view(np.uint32), np.ascontiguousarray(want).view(np.uint32))
        assert np.array_equal(q[:, :k].float().cpu().numpy(), rq)
        assert not q.view(torch.uint8)[:, k:].any()


def test_quantize_special_blocks(vq):
    x = torch.randn((12, 300), generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 17] = float("nan")
    x[2, 299] = float("inf")
    x[3, 130] = -float("inf")
    x[4] *= 1e-38          # subnormal and barely normal values: the scales are subnormal
    x[5] = 0
    x[5, 5] = 1e-45        # the scale rounds to zero
    x[6] *= 1e37           # large, finite
    x[7] = 0
    x[7, 1], x[7, 2], x[7, 3] = 448.0, 17.0, 2.0 ** -10   # ties: 17 lies between 16 and 18, 2^-10 between 0 and 2^-9
    x[8] *= 2e-33
    x[9] = -0.0
    x[10] = torch.linspace(-448, 448, 300)
    q, s = vq.f8_quantize(x.cuda())
    rq, rs = f8ref.quantize(x.numpy().astype(np.float64))
    s = s.t().cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(rs)) and np.array_equal(s[~np.isnan(rs)], rs[~np.isnan(rs)])
    assert np.array_equal(q[:, :300].float().cpu().numpy(), rq)


def test_quantize_views(vq):
    big = _x(np.random.default_rng(3), 50, 700, "bf16")
    for x in (big[:, 100:401], big[::3, :130], big[7:8, 1:600]):
        for rows in (1, 128):
            q, s = vq.f8_quantize(x, rows)
            rq, rs = f8ref.quantize(f8ref.widen(x), rows)
            assert np.array_equal(q[:, :x.shape[1]].float().cpu().numpy(), rq)
            assert np.array_equal(s.cpu().numpy(), rs.T if rows == 1 else rs)


# every way of the product, on both sides of its edges
SHAPES = [(1, 1, 1), (1, 16, 128), (1, 17, 129), (1, 128, 1000), (1, 5003, 4099), (1, 20000, 300), (1, 130, 20000), (2, 64, 64),
          (3, 777, 1030), (4, 4096, 4096), (5, 200, 4096), (16, 16, 8192), (16, 7001, 700), (17, 64, 128), (17, 65, 9000),
          (37, 5003, 4099), (64, 257, 1100), (65, 128, 128), (77, 2056, 5001), (128, 1024, 8192), (129, 129, 129), (200, 3000, 777),
          (256, 256, 256), (300, 6500, 1000), (513, 2050, 385), (2049, 6500, 260), (513, 7225, 130), (200, 8229, 385), (200, 8212, 1000), (130, 5485, 1000),
          (200, 8198, 130), (1, 83, 9000), (33, 8212, 130), (3, 28672, 256), (385, 900, 9000), (130, 903, 20000), (385, 65, 20000)]


def _exact_ints(vq, g, m, n, k, halves=1):
    """Operands whose products are exact in fp32 in every order: whole numbers up to 4, scales that are powers of two."""
    q, w = g.integers(-4, 5, (m, k)), g.integers(-4, 5, (halves * n, k))
    s = np.exp2(g.integers(-2, 3, (f8ref.blocks(k), m))).astype(np.float32)
    sw = np.exp2(g.integers(-2, 3, (halves * f8ref.blocks(n), f8ref.blocks(k)))).astype(np.float32)
    dev = lambda v: vq.f8_pad(torch.from_numpy(v.astype(np.float32)).to(E4)).cuda()
    x64 = q * f8ref.spread(s.T, m, k, 1)
    w64 = w * np.concatenate([f8ref.spread(p, n, k, 128) for p in np.split(sw, halves)])
    return dev(q), torch.from_numpy(s).cuda(), dev(w), torch.from_numpy(sw).cuda(), x64, w64


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_exact(vq, m, n, k):
    # |sum| <= 16 * 16 K in steps of 1 / 16: 24 bits hold it up to K = 2^12; longer ones stay below it in their sums' spread
    g = np.random.default_rng([m, n, k, 1])
    q, s, w, sw, x64, w64 = _exact_ints(vq, g, m, n, k)
    y64 = x64 @ w64.T
    assert np.abs(x64).max() <= 16 and np.abs(y64).max() < 2 ** 19
    for ws in (None, _ws(vq.f8_gemm_workspace_bytes(m, n, k))):
        for out in ("f32", "bf16"):
            print("product", m, n, k, ws is not None, out, flush=True)
            y = vq.f8_gemm(q, s, w, sw, None, k, ws=ws, y_dtype=DT[out])
            torch.cuda.synchronize()
            assert torch.equal(y.cpu(), torch.from_numpy(y64.astype(np.float32)).to(DT[out]))


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dt,out,bias", [("bf16", "bf16", False), ("f16", "f32", True)])
def test_linear(vq, m, n, k, dt, out, bias):
    g = np.random.default_rng([m, n, k])
    x = _x(g, m, k, dt)
    w, sw, w64 = _w(vq, g, n, k)
    b = torch.from_numpy(g.standard_normal(n).astype(np.float16)).cuda() if bias else None
    ref, bound = f8ref.product(_tokens(x), w64, f8ref.widen(b) if bias else None, narrow=out != "f32")
    print("linear", m, n, k, dt, out, flush=True)
    ws = _ws(vq.f8_linear_workspace_bytes(m, n, k))
    y = vq.f8_linear(x, w, sw, b, ws, y_dtype=DT[out])
    torch.cuda.synchronize()
    f8ref.check(y, ref, bound, out)
    assert torch.equal(y, vq.f8_linear(x, w, sw, b, ws, y_dtype=DT[out]))  # equal calls, equal bits
    # the two calls that it stands for, with and without a workspace
    q, s = vq.f8_quantize(x)
    for ws in (None, _ws(vq.f8_gemm_workspace_bytes(m, n, k))):
        f8ref.check(vq.f8_gemm(q, s, w, sw, b, k, ws=ws, y_dtype=DT[out]), ref, bound, out)


@pytest.mark.parametrize("m,n,k", [s for s in SHAPES if s[1] * s[2] <= 6500 * 1100])
def test_gated(vq, m, n, k):
    g = np.random.default_rng([m, n, k, 2])
    x = _x(g, m, k, "bf16")
    w, sw, w64 = _w(vq, g, n, k, halves=2)
    b = torch.from_numpy(g.standard_normal(2 * n).astype(np.float16)).cuda() if n % 2 else None
    t, b64 = _tokens(x), None if b is None else f8ref.widen(b)
    half = lambda v, i: None if v is None else v[i * n:(i + 1) * n]
    g64 = lambda narrow: f8ref.gate(*(v for i in (0, 1) for v in f8ref.product(t, half(w64, i), half(b64, i), narrow=narrow)))
    ref, bound = g64(False)
    print("gated", m, n, k, flush=True)
    y = vq.f8_linear(x, w, sw, b, _ws(vq.f8_linear_workspace_bytes(m, n, k, True)), gated=True, y_dtype=torch.float32)
    f8ref.check(y, ref, bound, "f32")
    q, s = vq.f8_quantize(x)
    f8ref.check(vq.f8_gemm(q, s, w, sw, b, k, gated=True, y_dtype=torch.bfloat16), *g64(True), "bf16")


@pytest.mark.parametrize("m,d,i,dt", [(1, 64, 100, "f16"), (1, 4096, 1000, "bf16"), (1, 200, 20000, "bf16"), (2, 300, 777, "f32"),
                                      (4, 512, 1024, "bf16"), (6, 1000, 129, "f16"), (30, 260, 1500, "bf16"),
                                      (77, 2056, 501, "f16"), (300, 128, 640, "bf16"), (513, 256, 9300, "bf16"),
                                      (700, 136, 10000, "f16"), (2100, 72, 3001, "bf16")])
def test_mlp(vq, m, d, i, dt):
    g = np.random.default_rng([m, d, i])
    x = _x(g, m, d, dt)
    w_in, s_in, in64 = _w(vq, g, i, d, halves=2)
    w_out, s_out, out64 = _w(vq, g, d, i)
    t = _tokens(x)
    ws = _ws(vq.f8_mlp_workspace_bytes(m, d, i))
    for out, narrow in (("bf16", (True, True)), ("f16", (False, True)), ("f32", (False, False))):
        print("mlp", m, d, i, out, flush=True)
        h, dh = f8ref.gate(*(v for w in (in64[:i], in64[i:]) for v in f8ref.product(t, w, narrow=narrow[0])))
        h, dh = f8ref.cut(h, dh)
        ref, bound = f8ref.product(h, out64, dx=dh, narrow=narrow[1])
        y = vq.f8_mlp(x, w_in, s_in, w_out, s_out, i, ws, y_dtype=DT[out])
        torch.cuda.synchronize()
        f8ref.check(y, ref, bound, out)
    assert torch.equal(y, vq.F8MLP(w_in[:, :d], s_in, w_out[:, :i], s_out)(x, torch.float32))


def test_rows_behind_the_last_are_left(vq):
    """Outputs of M rows in a longer buffer; columns past N in the 8-bit hidden rows are zero by their effect above."""
    g = np.random.default_rng(5)
    for m, n, k in ((3, 70, 200), (40, 70, 200), (70, 200, 129), (300, 6500, 200)):
        x = _x(g, m, k, "bf16")
        w, sw, _ = _w(vq, g, n, k)
        y = torch.full((m + 3, n), 7.0, device="cuda")
        vq.f8_linear(x, w, sw, None, _ws(vq.f8_linear_workspace_bytes(m, n, k)), out=y[:m])
        assert bool((y[m:] == 7).all()) and not bool((y[:m] == 7).all())


@pytest.mark.parametrize("m", [1, 3, 20, 70, 300])
def test_bad_values_stay_in_their_row(vq, m):
    """A token with a NaN or an infinity has NaN outputs, no other token's change; a NaN weight hits its own channel."""
    n, k = 6600, 300
    g = np.random.default_rng(m)
    x = _x(g, m, k, "f16")
    w, sw, _ = _w(vq, g, n, k)
    lay = vq.F8Linear(w[:, :k], sw)
    y = lay(x, torch.float32)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2 = x.clone()
        x2[m // 2, 140] = bad
        y2 = lay(x2, torch.float32)
        assert bool(torch.isnan(y2[m // 2]).all())
        rest = [r for r in range(m) if r != m // 2]
        assert torch.equal(y2[rest], y[rest])
    w.view(torch.uint8)[33, 299] = 0x7F
    y2 = lay.__class__(w[:, :k], sw)(x, torch.float32)
    assert bool(torch.isnan(y2[:, 33]).all())
    keep = [c for c in range(n) if c != 33]
    assert torch.equal(y2[:, keep], y[:, keep])


def test_layers(vq):
    g = np.random.default_rng(9)
    x = _x(g, 6, 500, "bf16")
    dense = torch.from_numpy(g.standard_normal((300, 500)).astype(np.float32) * 0.05).cuda()
    lay = vq.F8Linear.from_weight(dense)
    wq, wsc = f8ref.quantize(f8ref.widen(dense), 128)
    w64 = wq * f8ref.spread(wsc, 300, 500, 128)
    ref, bound = f8ref.product(_tokens(x), w64)
    f8ref.check(lay(x), *f8ref.product(_tokens(x), w64, narrow=True), "bf16")
    assert lay(x.reshape(2, 3, 500)).shape == (2, 3, 300)
    assert torch.equal(lay(x.reshape(2, 3, 500)).reshape(6, 300), lay(x))
    assert lay(x[:0]).shape == (0, 300)
    f8ref.check(lay.forward_f8(*vq.f8_quantize(x), torch.float32), ref, bound, "f32")
    # strided, expanded and transposed tokens
    wide = _x(g, 6, 1200, "bf16")
    assert torch.equal(lay(wide[:, 7:507]), lay(wide[:, 7:507].contiguous()))
    one = x[:1].expand(4, 500)
    assert torch.equal(lay(one), lay(one.contiguous()))
    tr = _x(g, 500, 6, "bf16").t()
    assert torch.equal(lay(tr), lay(tr.contiguous()))
    up, out = (torch.from_numpy(g.standard_normal(s).astype(np.float32) * 0.05).cuda() for s in ((300, 500), (500, 300)))
    mlp = vq.F8MLP.from_weights(dense, up, out)
    assert mlp(x.reshape(3, 2, 500)).shape == (3, 2, 500)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    xd, (gd, ud, od) = x.double(), (t.double() for t in (dense, up, out))
    gate, u = xd @ gd.t().contiguous(), xd @ ud.t().contiguous()
    # e4m3 rounds by at most 2^-4, evenly spread over a step by a third of that: four roundings on the way, two of them of
    # factors of one product: 2 * 0.036 a product, under 0.1 for the two in a row and their gate
    assert rel(mlp(x), (gate / (1 + torch.exp(-gate)) * u) @ od.t().contiguous()) < 0.1
    with pytest.raises(ValueError):
        lay(x[:, :499])
    with pytest.raises(ValueError):
        vq.F8Linear(torch.zeros((4, 8), dtype=E4, device="cuda"), torch.zeros((1, 2), device="cuda"))
    with pytest.raises(TypeError):
        lay(x.to(torch.float64))
    with pytest.raises(vq.VQError):
        vq.f8_quantize(torch.zeros((1, 65537), device="cuda"))


def test_streams_and_graphs(vq):
    """On another stream, and captured: every replay gives what the eager call gives on the inputs of the moment."""
    g = np.random.default_rng(12)
    mlp = vq.F8MLP.from_weights(*(torch.from_numpy(g.standard_normal(s).astype(np.float32) * 0.05).cuda()
                                  for s in ((640, 256), (640, 256), (256, 640))))
    for m in (1, 5, 40, 300):
        x = _x(g, m, 256, "bf16")
        want = mlp(x)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            y = mlp(x)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        xs = x.clone()
        with torch.cuda.graph(graph):
            ys = mlp(xs)
        for it in range(3):
            xs.copy_(x * (it + 1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(ys, mlp(x * (it + 1)))
