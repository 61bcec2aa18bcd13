"""GPU parity of vq_rotate_heads against the 64-bit form in f8ref.rotate, within its bound and half an ulp of the output."""
import math

import numpy as np
import pytest

import f8ref

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


def _rand(g, shape, dt="f32", spread=1.0):
    return torch.from_numpy((g.standard_normal(shape) * spread).astype(np.float32)).to(DT[dt]).cuda()


def _freqs(vq, rot, base, scaling=None):
    return vq.rope_frequencies(rot, base, scaling)[0]


def _case(vq, b, t, hq, hk, d, rot, start, inter, norm, dt="bf16", out=None, bias=False, wide=True, far=1 << 20, wdt="f32"):
    g = np.random.default_rng([b, t, hq, d, rot])
    qkv = _rand(g, (b, t, (hq + 2 * hk) * d), dt)
    q, k = qkv[..., :hq * d].view(b, t, hq, d), qkv[..., hq * d:(hq + hk) * d].view(b, t, hk, d)
    pos = torch.from_numpy(g.integers(0, far, (b, t))).to(torch.int64 if wide else torch.int32).cuda()
    scaling = {"kind": "yarn", "factor": 8.0, "length": 4096} if rot > 2 else None
    rotary = vq.Rotary(rot, 10000.0, start, inter, scaling) if rot else None
    vec = lambda on: _rand(g, d, wdt) if on else None
    kw = dict(q_weight=vec(norm != "none"), k_weight=vec(norm != "none"), q_bias=vec(bias), k_bias=vec(bias))
    print("heads", b, t, hq, hk, d, rot, start, inter, norm, dt, out, flush=True)
    got = vq.rotate_heads(q, k, pos, rotary, norm=norm, out_dtype=DT[out] if out else None, weight_offset=0.5, eps=1e-5, **kw)
    torch.cuda.synchronize()
    for x, y, w, c in ((q, got[0], kw["q_weight"], kw["q_bias"]), (k, got[1], kw["k_weight"], kw["k_bias"])):
        f = lambda v: None if v is None else f8ref.widen(v)
        ref, bound = f8ref.rotate(f8ref.widen(x), pos.cpu().numpy(), _freqs(vq, rot, 10000.0, scaling) if rot else [], rot, start,
                                  inter, rotary.scale if rot else 1.0, norm, f(w), f(c), 1e-5, 0.5)
        f8ref.check(y, ref, bound, out or dt)
    return got


# heads of every size and part: whole items, short ones, parts that begin and end anywhere, two items a lane
@pytest.mark.parametrize("d,rot,start", [(128, 128, 0), (64, 64, 0), (128, 64, 64), (192, 64, 128), (256, 256, 0), (80, 80, 0),
                                         (96, 32, 0), (112, 56, 3), (1, 0, 0), (2, 2, 0), (7, 4, 1), (8, 6, 2), (16, 16, 0),
                                         (33, 30, 1), (130, 2, 127), (576, 64, 512), (1000, 500, 200), (1024, 1024, 0),
                                         (1023, 1022, 1), (1024, 0, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
def test_heads(vq, d, rot, start, inter, norm):
    _case(vq, 2, 3, 5, 2, d, rot, start, inter, norm, bias=norm == "layer")


@pytest.mark.parametrize("dt,out", [("f16", None), ("f32", None), ("bf16", "f32"), ("f32", "bf16"), ("f16", "bf16")])
@pytest.mark.parametrize("norm", ["none", "rms"])
def test_types(vq, dt, out, norm):
    _case(vq, 1, 5, 4, 4, 128, 128, 0, False, norm, dt, out, wide=False, wdt=dt)
    _case(vq, 3, 2, 6, 1, 72, 36, 5, True, norm, dt, out, bias=norm != "none", wdt=dt)


# one token to many, few heads and many: both sides of every split of the work
@pytest.mark.parametrize("b,t,hq,hk", [(1, 1, 1, 1), (1, 1, 64, 8), (16, 1, 32, 8), (1, 1, 300, 7), (5, 1, 1, 1), (1, 1023, 3, 1),
                                       (1, 1024, 3, 1), (2, 513, 9, 3), (3, 400, 40, 8), (1025, 1, 2, 2)])
def test_sizes(vq, b, t, hq, hk):
    _case(vq, b, t, hq, hk, 64, 64, 0, False, "rms")
    _case(vq, b, t, hq, hk, 40, 12, 20, True, "none", "f16")


def test_far_positions(vq):
    """The angle of a far position is that of fp64: in fp32 it would be off by radians."""
    g = np.random.default_rng(4)
    x = _rand(g, (7, 2, 64))
    rotary = vq.Rotary(64, 500000.0)
    pos = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), (1 << 40) + 12345, 1 << 52], device="cuda")
    ref, bound = f8ref.rotate(f8ref.widen(x)[None], pos.cpu().numpy()[None], _freqs(vq, 64, 500000.0), 64)
    # the frequencies are given in turns, two roundings from radians: 2^-52 of the angle more
    ang = np.abs(pos.cpu().numpy()[:, None] * np.asarray(_freqs(vq, 64, 500000.0)))
    more = np.concatenate([ang, ang], axis=1)[None, :, None] * 2.0 ** -51 * 2 * np.abs(f8ref.widen(x)).max()
    near = bound + np.minimum(more, 100.0)
    f8ref.check(vq.rotate_heads(x, None, pos, rotary)[0][None], ref, near, "f32")
    assert float(near[0, :5].max()) < 1e-3  # which still says something up to 2^31
    # back again, in fp32
    y = vq.rotate_heads(x, None, pos[:5], rotary)[0] if x.shape[0] == 5 else vq.rotate_heads(x[:5], None, pos[:5], rotary)[0]
    z = vq.rotate_heads(y, None, -pos[:5], rotary)[0]
    assert float((z - x[:5]).abs().max()) <= 16 * f8ref.E * 2 * float(x.abs().max())
    assert torch.equal(vq.rotate_heads(x[:1], None, pos[:1], rotary)[0], x[:1])  # position 0


def test_views_and_places(vq):
    """Strides of any kind, positions shared by the batches, outputs in place and into views; what is beside them is left."""
    g = np.random.default_rng(8)
    b, t, hq, hk, d = 2, 5, 4, 2, 64
    rotary = vq.Rotary(d, interleaved=True)
    q, k = _rand(g, (b, t, hq, d), "bf16"), _rand(g, (b, t, hk, d), "bf16")
    w = _rand(g, d)
    pos = torch.arange(t, device="cuda") + 100
    kw = dict(norm="rms", q_weight=w, k_weight=w)
    want = vq.rotate_heads(q, k, pos, rotary, **kw)
    same = lambda got, w=want: all(torch.equal(x, y) for x, y in zip(got, w))
    assert same(vq.rotate_heads(q, k, pos.expand(b, t).contiguous(), rotary, **kw))
    assert same(vq.rotate_heads(q, k, pos.int(), rotary, **kw))
    # batch by batch
    for i in range(b):
        assert same(vq.rotate_heads(q[i], k[i], pos, rotary, **kw), [x[i] for x in want])
    # [batch, heads, tokens, dim] in memory
    qt, kt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k))
    assert same(vq.rotate_heads(qt, kt, pos, rotary, **kw))
    out = [torch.empty_like(x.transpose(1, 2).contiguous()).transpose(1, 2) for x in (q, k)]
    assert same(vq.rotate_heads(q, k, pos, rotary, q_out=out[0], k_out=out[1], **kw)) and same(out)
    # odd strides and an unaligned start
    odd = torch.full((b, t, hq + 1, d + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    view = odd[:, :, :hq, 1:d + 1]
    view.copy_(q)
    got = vq.rotate_heads(view, None, pos, rotary, norm="rms", q_weight=w, q_out=view)  # in place
    assert got[1] is None and got[0] is view and torch.equal(view, want[0])
    assert bool((odd[:, :, hq] == 9).all()) and bool((odd[..., 0] == 9).all()) and bool((odd[..., d + 1:] == 9).all())
    # expanded inputs
    one = q[:, :1].expand(b, t, hq, d)
    assert torch.equal(vq.rotate_heads(one, None, pos, rotary)[0], vq.rotate_heads(one.contiguous(), None, pos, rotary)[0])
    # nothing to do
    assert vq.rotate_heads(q[:0], k[:0], pos, rotary)[0].shape == (0, t, hq, d)
    assert vq.rotate_heads(q[:, :0], k[:, :0], pos[:0], rotary)[1].shape == (b, 0, hk, d)
    assert vq.rotate_heads(q[:, :, :0], k, pos, rotary, **kw)[0].shape == (b, t, 0, d)
    # a norm alone, and nothing at all
    alone = vq.rotate_heads(q, k, None, None, **kw)
    ref, bound = f8ref.rotate(f8ref.widen(q), np.zeros((b, t)), [], 0, norm="rms", w=f8ref.widen(w))
    f8ref.check(alone[0], ref, bound, "bf16")
    assert torch.equal(vq.rotate_heads(q, None, None, None)[0], q)


def test_special_values(vq):
    """A zero head, and heads with an infinity or a NaN: no other head changes; what is not rotated passes as it is."""
    g = np.random.default_rng(2)
    x = _rand(g, (3, 4, 64))
    rotary = vq.Rotary(32, start=16)
    pos = torch.tensor([3, 4, 5], device="cuda")
    y = vq.rotate_heads(x, None, pos, rotary, norm="rms")[0]
    x2 = x.clone()
    x2[0, 0] = 0
    x2[1, 1, 5] = float("inf")
    x2[2, 2, 20] = float("nan")
    y2 = vq.rotate_heads(x2, None, pos, rotary, norm="rms")[0]
    assert not bool(y2[0, 0].any()) and bool(torch.isnan(y2[2, 2]).all())
    keep = torch.ones((3, 4), dtype=torch.bool)
    keep[0, 0] = keep[1, 1] = keep[2, 2] = False
    assert torch.equal(y2[keep], y[keep])
    z = vq.rotate_heads(x2, None, pos, rotary)[0]
    assert torch.equal(z[..., :16], x2[..., :16]) and torch.equal(z[..., 48:].isnan(), x2[..., 48:].isnan())
    assert bool(torch.isnan(z[2, 2, 20])) and bool(torch.isnan(z[2, 2, 36])) and int(torch.isnan(z).sum()) == 2


def test_refusals(vq):
    x = torch.zeros((2, 3, 4, 8), device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    r = vq.Rotary(8)
    for call in (lambda: vq.rotate_heads(x.transpose(2, 3), None, pos, r),             # heads not contiguous
                 lambda: vq.rotate_heads(x[0, 0], None, pos, r), lambda: vq.rotate_heads(x, x[0], pos, r),
                 lambda: vq.rotate_heads(x, x[:, :2], pos, r),                          # other tokens
                 lambda: vq.rotate_heads(x, x.half(), pos, r),                          # other type
                 lambda: vq.rotate_heads(x, None, pos[:2], r),                          # other positions
                 lambda: vq.rotate_heads(x[0], None, pos[None], r),
                 lambda: vq.rotate_heads(x, None, pos, vq.Rotary(8, start=1)),          # past the head
                 lambda: vq.rotate_heads(x, None, pos, r, q_out=x[:, :2]),
                 lambda: vq.rotate_heads(x, None, pos, r, k_weight=x[0, 0, 0]),
                 lambda: vq.rotate_heads(x, None, pos, r, norm="rms", q_weight=x[0, 0, 0, :7])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        vq.rotate_heads(x, None, pos.float(), r)
    with pytest.raises(TypeError):
        vq.rotate_heads(x.double(), None, pos, r)
    for call in (lambda: vq.rotate_heads(x, None, pos, r, q_weight=x[0, 0, 0]),                    # weights without a norm
                 lambda: vq.rotate_heads(x, None, pos, r, q_out=x[:1].expand(2, 3, 4, 8)),         # outputs over each other
                 lambda: vq.rotate_heads(x[:1].expand(2, 3, 4, 8), None, pos, r, q_out=x)):        # in place with other strides
        with pytest.raises(vq.VQError):
            call()


def test_streams_and_graphs(vq):
    g = np.random.default_rng(6)
    rotary, w = vq.Rotary(128), _rand(g, 128)
    q, k = _rand(g, (9, 8, 128), "bf16"), _rand(g, (9, 2, 128), "bf16")
    pos = torch.arange(9, device="cuda")
    run = lambda: vq.rotate_heads(q, k, pos, rotary, norm="rms", q_weight=w, k_weight=w)
    want = run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run()
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for it in range(3):
        pos.add_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, run()))


def test_frequencies_meet_their_formula(vq):
    """One pair, one position: cos and sin of the angle in radians."""
    r = vq.Rotary(2, 10000.0)
    x = torch.tensor([[[1.0, 0.0]]], device="cuda")
    y = vq.rotate_heads(x, None, torch.tensor([1], device="cuda"), r)[0].flatten().tolist()
    assert abs(y[0] - math.cos(1.0)) < 2e-7 and abs(y[1] - math.sin(1.0)) < 2e-7
