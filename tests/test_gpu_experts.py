"""GPU parity of the expert operators (vq_expert_plan, vq_q8_gemm_grouped, vq_expert_combine, vq_q8_experts) against
64-bit references: the plan's integers equal a stable sort's, each product within its derived bound, and the whole
layer equal, bit for bit, to its parts called one by one.
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


def _ids(g, t, e, top, how="skewed"):
    if how == "one":        # every token picks the same experts
        return np.tile(np.arange(top)[::-1], (t, 1)).astype(np.int32)
    score = g.standard_normal((t, e)) + g.standard_normal(e)[None, :]
    ids = np.argsort(-score, axis=1)[:, :top].astype(np.int32)
    if how == "dropped":    # some pairs belong to no expert here
        ids[g.random(ids.shape) < 0.3] = -1
        ids[g.random(ids.shape) < 0.1] = e + 3
    return ids


def _layer(g, e, d, i):
    w = lambda n, k: np.clip(np.rint(g.standard_normal((e, n, k)) * 40), -127, 127).astype(np.int8)
    s = lambda n: g.uniform(0.5, 1.5, (e, n)).astype(np.float32) * np.float32(1.0 / (40 * d ** 0.5))
    return w(2 * i, d), s(2 * i), w(d, i), s(d)


def _x(g, t, d, dt):
    x = g.standard_normal((t, d))
    x[:, g.random(d) < 0.01] *= 10
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt]).cuda()


cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("t,e,top", [(1, 1, 1), (1, 8, 2), (7, 64, 4), (333, 64, 4), (1024, 3, 3), (1025, 7, 1),
                                     (4096, 8, 2), (3000, 300, 8), (5, 4096, 2), (40000, 16, 2)])
@pytest.mark.parametrize("how", ["skewed", "one", "dropped"])
def test_plan(vq, t, e, top, how):
    ids = _ids(np.random.default_rng([t, e, top]), t, e, top, how)
    off, rows, pos = vq.expert_plan(cu(ids), e)
    ro, rr, rp = q8ref.plan(ids, e)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(rows.cpu().numpy()[:ro[-1]], rr)
    assert np.array_equal(pos.cpu().numpy(), rp)


def test_plan_of_nothing(vq):
    off, rows, pos = vq.expert_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert not off.any() and rows.numel() == 0 and pos.shape == (0, 2)
    off, rows, pos = vq.expert_plan(torch.full((3, 2), -7, dtype=torch.int32, device="cuda"), 5)
    assert not off.any() and bool((pos == -1).all())


CASES = [(1, 8, 2, 256, 384), (3, 2, 1, 130, 65), (40, 64, 4, 200, 100), (100, 4, 2, 129, 257), (333, 6, 3, 512, 160),
         (150, 1, 1, 300, 140), (500, 3, 2, 640, 200)]


@pytest.mark.parametrize("t,e,top,d,i", CASES)
@pytest.mark.parametrize("how", ["skewed", "one", "dropped"])
def test_grouped_products(vq, t, e, top, d, i, how):
    print("grouped", t, e, top, d, i, how, flush=True)
    g = np.random.default_rng([t, e, top, d, i])
    top = min(top, e)
    ids = _ids(g, t, e, top, how)
    off, rows, pos = q8ref.plan(ids, e)
    w_in, s_in, w_out, s_out = _layer(g, e, d, i)
    b_in = (g.standard_normal((e, 2 * i)) * 0.2).astype(np.float16)
    r = t * top
    q, s = vq.q8_quantize(_x(g, t, d, "f16"))
    qn, sn = q[:, :d].cpu().numpy(), s.cpu().numpy()
    rows_d = torch.zeros(r, dtype=torch.int32, device="cuda")
    rows_d[:len(rows)] = cu(rows)
    wi, wo = vq.q8_pad(cu(w_in)), vq.q8_pad(cu(w_out))
    keep = int(off[-1])
    for bias in (None, b_in):
        for gated in (True, False):
            for out in ("f32", "bf16"):
                y = torch.full((r, i if gated else 2 * i), 7.0, dtype=DT[out], device="cuda")
                vq.q8_gemm_grouped(cu(off), rows_d, q, s, wi, cu(s_in), None if bias is None else cu(bias), d, r,
                                   gated=gated, out=y)
                assert bool((y[keep:] == 7.0).all())          # rows past the last group are left alone
                for ex in range(e):
                    a, b = off[ex], off[ex + 1]
                    if a == b:
                        continue
                    f = q8ref.gated if gated else q8ref.product
                    ref, bound = f(qn[rows[a:b]], sn[rows[a:b]], w_in[ex], s_in[ex], None if bias is None else bias[ex])
                    q8ref.check(y[a:b], ref, bound, out)
    # rows in sorted order already: no gather
    h = torch.randn((r, i), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    hq, hs = vq.q8_quantize(h)
    z = vq.q8_gemm_grouped(cu(off), None, hq, hs, wo, cu(s_out), None, i, r)
    for ex in range(e):
        a, b = off[ex], off[ex + 1]
        if a < b:
            ref, bound = q8ref.product(hq[a:b, :i].cpu().numpy(), hs[a:b].cpu().numpy(), w_out[ex], s_out[ex])
            q8ref.check(z[a:b], ref, bound, "f32")


@pytest.mark.parametrize("gated", [True, False])
def test_grouped_many_tiles(vq, gated):
    """Groups long enough for 256-row tiles, and enough tiles for several rounds over the CUs, the last one in halves."""
    g = np.random.default_rng(77)
    t, e, top, d, n = 2500, 5, 2, 70, 4000
    ids = _ids(g, t, e, top)
    off, rows, pos = q8ref.plan(ids, e)
    w = np.clip(np.rint(g.standard_normal((e, 2 * n, d)) * 40), -127, 127).astype(np.int8)
    sw = g.uniform(0.5, 1.5, (e, 2 * n)).astype(np.float32) * np.float32(3e-3)
    q, s = vq.q8_quantize(_x(g, t, d, "bf16"))
    y = vq.q8_gemm_grouped(cu(off), cu(rows), q, s, vq.q8_pad(cu(w)), cu(sw), None, d, t * top, gated=gated)
    qn, sn = q[:, :d].cpu().numpy(), s.cpu().numpy()
    for ex in range(e):
        a, b = off[ex], off[ex + 1]
        ref, bound = (q8ref.gated if gated else q8ref.product)(qn[rows[a:b]], sn[rows[a:b]], w[ex], sw[ex])
        q8ref.check(y[a:b], ref, bound, "f32")


def test_groups_outside_the_buffer_are_bounded(vq):
    """Offsets and rows that no plan wrote: nothing is read or written outside the buffers that were given."""
    g = np.random.default_rng(5)
    w_in, s_in, _, _ = _layer(g, 3, 64, 32)
    q, s = vq.q8_quantize(_x(g, 6, 64, "f32"))
    for off, rows in (([-5, 2, 4, 1000], [0, 1, 2, 3, 4, 5]), ([3, 1, 6, 2], [9, -1, 5, 70000, 0, 2])):
        guard = torch.full((10, 32), 7.0, device="cuda")
        vq.q8_gemm_grouped(cu(np.array(off, np.int32)), cu(np.array(rows, np.int32)), q, s, vq.q8_pad(cu(w_in)),
                           cu(s_in), None, 64, 6, gated=True, out=guard[2:8])
        torch.cuda.synchronize()
        assert bool((guard[:2] == 7.0).all()) and bool((guard[8:] == 7.0).all())
    # the same with the large tiles: groups that overlap ask for more tiles than the launch holds
    rows = torch.zeros(900, dtype=torch.int32, device="cuda")
    for off in ([0, 900, 5, 900], [900, 0, 900, 100], [-2 ** 31, 2 ** 31 - 1, -1, 2 ** 31 - 1]):
        guard = torch.full((904, 32), 7.0, device="cuda")
        vq.q8_gemm_grouped(cu(np.array(off, np.int64).astype(np.int32)), rows, q, s, vq.q8_pad(cu(w_in)), cu(s_in),
                           None, 64, 900, gated=True, out=guard[2:902])
        torch.cuda.synchronize()
        assert bool((guard[:2] == 7.0).all()) and bool((guard[902:] == 7.0).all())


@pytest.mark.parametrize("t,top,n", [(1, 1, 1), (3, 2, 5), (40, 4, 130), (300, 2, 1027), (2, 8, 4096)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_combine(vq, t, top, n, out):
    g = np.random.default_rng([t, top, n])
    z = g.standard_normal((t * top, n)).astype(np.float32)
    pos = g.permutation(t * top).astype(np.int32).reshape(t, top)
    pos[g.random(pos.shape) < 0.2] = -1
    p = g.random((t, top)).astype(np.float32)
    y = vq.expert_combine(cu(z), cu(pos), cu(p), y_dtype=DT[out])
    terms = np.where(pos[:, :, None] >= 0, p[:, :, None].astype(np.float64) * z[np.maximum(pos, 0)].astype(np.float64), 0)
    q8ref.check(y, terms.sum(1), (top + 1) * q8ref.E * np.abs(terms).sum(1) + 1e-40, out)


@pytest.mark.parametrize("t,e,top,d,i", CASES + [(1, 3, 1, 64, 4096), (700, 4, 2, 128, 200), (2, 40, 8, 1000, 333)])
@pytest.mark.parametrize("how,dt", [("skewed", "bf16"), ("one", "f16"), ("dropped", "f32")])
def test_whole_layer_equals_its_parts(vq, t, e, top, d, i, how, dt):
    print("experts", t, e, top, d, i, how, flush=True)
    g = np.random.default_rng([t, e, top, d, i, 1])
    top = min(top, e)
    ids = cu(_ids(g, t, e, top, how))
    p = cu(g.random((t, top)).astype(np.float32))
    w_in, s_in, w_out, s_out = (cu(v) for v in _layer(g, e, d, i))
    x = _x(g, t, d, dt)
    lay = vq.Q8Experts(w_in, s_in, w_out, s_out)
    y = lay(x, ids, p)
    off, rows, pos = vq.expert_plan(ids, e)
    q, s = vq.q8_quantize(x)
    r = t * top
    h = vq.q8_gemm_grouped(off, rows, q, s, lay.w_in, s_in, None, d, r, gated=True, out=torch.zeros((r, i), device="cuda"))
    hq, hs = vq.q8_quantize(h)
    z = vq.q8_gemm_grouped(off, None, hq, hs, lay.w_out, s_out, None, i, r, out=torch.zeros((r, d), device="cuda"))
    want = vq.expert_combine(z, pos, p, y_dtype=DT[dt])
    assert y.dtype == x.dtype and torch.equal(y, want)


@pytest.mark.parametrize("e,top,d,i", [(8, 2, 256, 384), (4, 4, 1000, 333), (12, 9, 128, 100), (6, 2, 130, 40000),
                                       (6, 2, 40000, 130), (2, 1, 1, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_token_layer(vq, e, top, d, i, dt):
    """One token: its own two launches, and more slots or longer rows than those take; ids of no expert among them."""
    g = np.random.default_rng([e, top, d, i])
    w_in, s_in, w_out, s_out = (cu(v) for v in _layer(g, e, d, i))
    lay = vq.Q8Experts(w_in, s_in, w_out, s_out)
    x, p = _x(g, 1, d, dt), cu(g.random((1, top)).astype(np.float32))
    full = _ids(g, 1, e, top)
    for drop in ((), (0,), tuple(range(top))):
        ids = full.copy()
        ids[0, list(drop)] = -1 if len(drop) == 1 else e
        y = lay(x, cu(ids), p, y_dtype=torch.float32)
        off, rows, pos = vq.expert_plan(cu(ids), e)
        q, s = vq.q8_quantize(x)
        h = vq.q8_gemm_grouped(off, rows, q, s, lay.w_in, s_in, None, d, top, gated=True,
                               out=torch.zeros((top, i), device="cuda"))
        hq, hs = vq.q8_quantize(h)
        z = vq.q8_gemm_grouped(off, None, hq, hs, lay.w_out, s_out, None, i, top, out=torch.zeros((top, d), device="cuda"))
        assert torch.equal(y, vq.expert_combine(z, pos, p)), drop
    assert not y.any()


def test_whole_layer_against_dense(vq):
    """One token at a time through its own experts' 64-bit products: close up to the 8-bit step of the hidden row."""
    g = np.random.default_rng(3)
    t, e, top, d, i = 9, 5, 2, 200, 150
    ids, p = _ids(g, t, e, top), g.random((t, top)).astype(np.float32)
    w_in, s_in, w_out, s_out = _layer(g, e, d, i)
    x = _x(g, t, d, "f32")
    y = q8ref.widen(vq.Q8Experts(cu(w_in), cu(s_in), cu(w_out), cu(s_out))(x, cu(ids), cu(p)))
    q, s = q8ref.quantize(q8ref.widen(x))
    for k in range(t):
        want, lim = np.zeros(d), np.zeros(d)
        for j in range(top):
            ex = ids[k, j]
            h, dh = q8ref.gated(q[k:k + 1], s[k:k + 1], w_in[ex], s_in[ex])
            hs = np.abs(h).max() / 127
            w64 = w_out[ex].astype(np.float64) * s_out[ex].astype(np.float64)[:, None]
            want += p[k, j] * (np.clip(np.rint(h / hs), -127, 127) * hs @ w64.T)[0]
            # a hidden value within its error of a tie may go either way: one step of it
            near = np.abs(np.abs(h / hs - np.floor(h / hs)) - 0.5) * hs <= 2 * dh + 1e-6 * hs
            lim += p[k, j] * ((near * hs) @ np.abs(w64).T)[0] + 1e-5 * np.abs(want)
        assert (np.abs(y[k] - want) <= lim + 1e-5 * np.abs(want).max()).all()


def test_nothing_and_everything_dropped(vq):
    g = np.random.default_rng(4)
    w_in, s_in, w_out, s_out = (cu(v) for v in _layer(g, 3, 64, 32))
    lay = vq.Q8Experts(w_in, s_in, w_out, s_out)
    none = lambda *s: torch.empty(s, device="cuda")
    assert lay(none(0, 64), none(0, 2).int(), none(0, 2)).shape == (0, 64)
    y = lay(_x(g, 4, 64, "f32"), torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), torch.ones((4, 2), device="cuda"))
    assert not y.any()


def test_graph_and_stream(vq):
    g = np.random.default_rng(6)
    t, e, top, d, i = 20, 6, 2, 256, 128
    lay = vq.Q8Experts(*(cu(v) for v in _layer(g, e, d, i)))
    st = torch.cuda.Stream()
    x, ids, p = _x(g, t, d, "bf16"), cu(_ids(g, t, e, top)), cu(g.random((t, top)).astype(np.float32))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        lay(x, ids, p)
    st.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        y = lay(x, ids, p)
    for k in range(3):
        g2 = np.random.default_rng([7, k])
        x.copy_(_x(g2, t, d, "bf16"))
        ids.copy_(cu(_ids(g2, t, e, top)))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, lay(x, ids, p)), k


def test_refusals(vq):
    g = np.random.default_rng(8)
    w_in, s_in, w_out, s_out = (cu(v) for v in _layer(g, 3, 64, 32))
    lay = vq.Q8Experts(w_in, s_in, w_out, s_out)
    x, p = _x(g, 4, 64, "f32"), torch.ones((4, 2), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        lay(x, ids.long(), p)
    with pytest.raises(ValueError):
        lay(x, ids, p[:3])
    with pytest.raises(TypeError):
        lay(x, ids, p.half())
    with pytest.raises(ValueError):
        lay(x[:, :63], ids, p)
    with pytest.raises(vq.VQError):
        vq.expert_plan(ids, 0)
    with pytest.raises(vq.VQError):
        vq.expert_plan(ids, 4097)
    with pytest.raises(ValueError):
        vq.expert_plan(ids[0], 3)
    q, s = vq.q8_quantize(x)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(vq.VQError):   # without a gather every sorted row needs a row of q
        vq.q8_gemm_grouped(off, None, q, s, lay.w_in, s_in, None, 64, 8, gated=True)
    with pytest.raises(ValueError):
        vq.q8_gemm_grouped(off[:3], None, q, s, lay.w_in, s_in, None, 64, 4)
    with pytest.raises(ValueError):
        vq.q8_gemm_grouped(off, ids.reshape(-1)[:3], q, s, lay.w_in, s_in, None, 64, 4)
