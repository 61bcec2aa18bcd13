"""vq_rotate_heads and its binding on the host (no GPU): the frequencies and every refusal, before anything is launched.
Pointers are made-up aligned addresses: nothing may be read through them."""
import ctypes
import math

import pytest

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


def _desc(vq, **kw):
    t = lambda *v: (ctypes.c_int64 * 3)(*v)
    f = dict(batch=2, tokens=3, q_heads=4, k_heads=2, dim=64, rot=64, start=0, interleaved=0, norm=1, x_dtype=0, y_dtype=0,
             w_dtype=2, positions_64=1, position_stride=3, q_strides=(768, 256, 64), k_strides=(384, 128, 64),
             q_out_strides=(768, 256, 64), k_out_strides=(384, 128, 64), scale=1.0, eps=1e-6, w_offset=0.0)
    f.update(kw)
    return vq.HeadsDesc(*[t(*v) if isinstance(v, tuple) else v for v in f.values()])


def test_refusals(vq):
    fn = vq.lib().vq_rotate_heads
    out = 1 << 21

    def call(q=P, k=P, pos=P, fr=P, w=(None,) * 4, yq=out, yk=out, **kw):
        return fn(ctypes.byref(_desc(vq, **kw)), q, k, pos, fr, *w, yq, yk, None)

    assert fn(None, P, P, P, P, P, P, P, P, P, P, None) == vq.VQ_ERR_NULL
    for kw in (dict(batch=-1), dict(tokens=-1), dict(q_heads=-1), dict(k_heads=65537), dict(dim=0), dict(dim=1025),
               dict(rot=63), dict(rot=66), dict(rot=-2), dict(start=-1), dict(start=1), dict(start=2 ** 31 - 1),
               dict(position_stride=-1), dict(q_strides=(-1, 256, 64)), dict(q_out_strides=(768, 256, 63)),
               dict(k_out_strides=(384, 0, 64)), dict(k_out_strides=(0, 128, 64)),
               dict(batch=2 ** 31 - 1, tokens=2 ** 31 - 1, q_strides=(0, 0, 0), k_strides=(0, 0, 0))):
        assert call(**kw) == vq.VQ_ERR_SHAPE, kw
    for kw in (dict(norm=3), dict(norm=-1), dict(interleaved=2), dict(positions_64=2), dict(x_dtype=7), dict(y_dtype=7),
               dict(w=(P, None, None, None), w_dtype=7), dict(norm=0, w=(P, None, None, None)),
               dict(norm=0, w=(None, None, None, P)),
               dict(yq=P, y_dtype=1), dict(yq=P, q_strides=(0, 256, 64))):  # in place, but not where it was read
        assert call(**kw) == vq.VQ_ERR_UNSUPPORTED, kw
    for kw in (dict(q=None), dict(k=None), dict(yq=None), dict(yk=None), dict(pos=None), dict(fr=None)):
        assert call(**kw) == vq.VQ_ERR_NULL, kw
    for kw in (dict(q=P + 1), dict(yk=out + 1), dict(x_dtype=2, q=P + 2), dict(pos=P + 4), dict(fr=P + 4),
               dict(w=(P + 2, None, None, None)), dict(w=(None, None, None, P + 1), w_dtype=0),
               dict(positions_64=0, pos=P + 2)):
        assert call(**kw) == vq.VQ_ERR_ALIGN, kw
    for kw in (dict(batch=0), dict(tokens=0), dict(q_heads=0, k_heads=0)):
        assert call(None, None, None, None, yq=None, yk=None, **kw) == vq.VQ_OK, kw


def test_frequencies(vq):
    f, s = vq.rope_frequencies(8, 10000.0)
    assert s == 1.0 and f == [1.0, 10000.0 ** -0.25, 10000.0 ** -0.5, 10000.0 ** -0.75]
    assert vq.rope_frequencies(0) == ([], 1.0)
    lin, s = vq.rope_frequencies(8, scaling={"kind": "linear", "factor": 4.0})
    assert s == 1.0 and lin == [v / 4 for v in f]
    ntk, s = vq.rope_frequencies(8, scaling={"kind": "ntk", "factor": 4.0})
    assert s == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4, rel_tol=1e-12)
    assert all(b / 4 <= a * (1 + 1e-12) and a <= b for a, b in zip(ntk, f))
    # the fastest pairs as they were, the slowest at 1 / s, in between in order
    base, dim, length = 10000.0, 128, 4096
    f, _ = vq.rope_frequencies(dim, base)
    yarn, s = vq.rope_frequencies(dim, base, {"kind": "yarn", "factor": 16.0, "length": length})
    assert math.isclose(s, 0.1 * math.log(16.0) + 1)
    lo = math.floor(dim * math.log(length / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(dim * math.log(length / (2 * math.pi)) / (2 * math.log(base)))
    for j in range(64):
        g = min(max((j - lo) / (hi - lo), 0), 1)
        assert math.isclose(yarn[j], f[j] / 16 * g + f[j] * (1 - g), rel_tol=1e-14)
    assert yarn[:lo + 1] == f[:lo + 1] and yarn[-1] == f[-1] / 16
    assert vq.rope_frequencies(dim, base, {"kind": "yarn", "factor": 16.0, "length": length, "scale": 1.5})[1] == 1.5
    bands, s = vq.rope_frequencies(dim, base, {"kind": "bands", "factor": 8.0, "length": length, "low": 1.0, "high": 4.0})
    assert s == 1.0
    for a, b in zip(bands, f):
        turns = length * b / (2 * math.pi)
        want = b if turns > 4 else b / 8 if turns < 1 else (turns - 1) / 3 * b + (4 - turns) / 3 * b / 8
        assert math.isclose(a, want, rel_tol=1e-12)
    lst, s = vq.rope_frequencies(4, scaling={"kind": "list", "factors": [1.0, 2.0], "scale": 1.25})
    assert lst == [1.0, 0.005] and s == 1.25


def test_frequency_refusals(vq):
    for a in ((7,), (-2,), (8, 0.0), (8, -1.0), (8, math.inf), (8, math.nan), (8, 1e4, {}), (8, 1e4, {"kind": "other"}),
              (8, 1e4, {"kind": "linear"}), (8, 1e4, {"kind": "linear", "factor": 0.0}),
              (8, 1e4, {"kind": "linear", "factor": 2.0, "length": 4}), (8, 1e4, {"kind": "yarn", "factor": 2.0}),
              (8, 1.0, {"kind": "yarn", "factor": 2.0, "length": 4}),
              (8, 1e4, {"kind": "bands", "factor": 2.0, "length": 4, "low": 4, "high": 4}),
              (8, 1e4, {"kind": "list", "factors": [1.0] * 3}), (8, 1e4, {"kind": "list", "factors": [1.0, 1.0, 1.0, -1.0]})):
        with pytest.raises(ValueError):
            vq.rope_frequencies(*a)
    with pytest.raises(ValueError):
        vq.Rotary(8, start=-1, device="cpu")


def test_rotary_object(vq):
    r = vq.Rotary(8, base=100.0, start=3, interleaved=True, scaling={"kind": "linear", "factor": 2.0}, device="cpu")
    f, s = vq.rope_frequencies(8, 100.0, {"kind": "linear", "factor": 2.0})
    assert (r.dim, r.start, r.interleaved, r.scale) == (8, 3, True, s)
    assert r.freqs.dtype == torch.float64 and r.freqs.tolist() == [v / (2 * math.pi) for v in f]


def test_binding_refuses_host_tensors(vq):
    x = torch.zeros((2, 4, 8))
    with pytest.raises(ValueError, match="device tensor"):
        vq.rotate_heads(x, None, torch.zeros(2, dtype=torch.int64), None)
    with pytest.raises(ValueError, match="norm must be"):
        vq.rotate_heads(x, None, None, None, norm="l2")


def test_one_tensor_written_over_the_other_is_refused(vq):
    """Queries and keys exchanged, or both written to one place: the heads of both are taken in any order."""
    fn = vq.lib().vq_rotate_heads
    k, out = 1 << 21, 1 << 22
    same = dict(k_heads=4, k_strides=(768, 256, 64), k_out_strides=(768, 256, 64))
    for yq, yk in ((k, P), (out, out), (k, out), (out, P)):
        assert fn(ctypes.byref(_desc(vq, **same)), P, k, P, P, *(None,) * 4, yq, yk, None) == vq.VQ_ERR_UNSUPPORTED, (yq, yk)


def test_rotation_needs_positions(vq, monkeypatch):
    monkeypatch.setattr(vq.heads, "_device", lambda t, what: -1)
    with pytest.raises(TypeError, match="positions"):
        vq.rotate_heads(torch.zeros((2, 4, 8)), None, None, vq.Rotary(8, device="cpu"))


def test_positions_of_any_batch_stride(vq, monkeypatch):
    """[batch, tokens] as views: expanded from one row, every other row, a column of a wider tensor; not every other token."""
    seen = []
    monkeypatch.setattr(vq.heads, "_device", lambda t, what: -1)
    monkeypatch.setattr(vq.heads, "_stream", lambda dev: 0)
    monkeypatch.setattr(vq.heads, "_launch", lambda fn, dev, desc, *a: seen.append((desc._obj, a[2])))
    rotary = vq.Rotary(8, device="cpu")
    q = torch.zeros((3, 5, 2, 8))
    wide = torch.arange(6 * 9).view(6, 9)
    for pos, stride in ((wide[0, :5], 0), (wide[0, :5].expand(3, 5), 0), (wide[::2, 2:7], 18), (wide[:3, :5].contiguous(), 5),
                        (wide[:3, :5].int(), 5)):
        vq.rotate_heads(q, None, pos, rotary)
        desc, p = seen.pop()
        assert (desc.position_stride, desc.positions_64, p) == (stride, int(pos.dtype is torch.int64), pos.data_ptr())
    for one, stride in ((wide[:3, 4:5], 9), (wide[4:5, :3].t(), 1)):  # a decode step: one position for each batch
        vq.rotate_heads(q[:, :1], None, one, rotary)
        assert seen.pop()[0].position_stride == stride
    vq.rotate_heads(q[:1], None, wide[2:3, :5], rotary)
    vq.rotate_heads(q[0, :1], None, wide[0, :1], rotary)
    seen.clear()
    for pos in (wide[:3, :9:2], wide[0, :9:2], wide[:5, :3].t(), wide[0, :1].expand(5), wide[:1, :5]):
        with pytest.raises(ValueError, match="positions"):
            vq.rotate_heads(q, None, pos, rotary)
    assert not seen
