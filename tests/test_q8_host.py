"""The 8-bit operators' C entry points on the host (no GPU): sizes, and every refusal, which has to come back before
anything is launched.  Pointers are made-up aligned addresses: nothing may be read through them."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def vq():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    g.lib()
    return g


P = 1 << 20  # a 256-byte aligned address that is nobody's
F16, F32, BAD = 0, 2, 7


def _size(f, *a):
    n = ctypes.c_size_t(12345)
    return f(*a, ctypes.byref(n)), n.value


def test_row_bytes(vq):
    for k, b in ((1, 128), (127, 128), (128, 128), (129, 256), (4099, 4224), (65536, 65536), (0, 0), (-5, 0)):
        assert vq.q8_row_bytes(k) == b


def test_workspace_sizes(vq):
    lib = vq.lib()
    for f, args in ((lib.vq_q8_gemm_workspace_bytes, (64, 128, 256)), (lib.vq_q8_linear_workspace_bytes, (64, 128, 256))):
        for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 65537)):
            assert _size(f, *bad)[0] == vq.VQ_ERR_SHAPE
        assert f(*args, None) == vq.VQ_ERR_NULL
        for zero in ((0, 128, 256), (64, 0, 256)):
            assert _size(f, *zero) == (0, 0)
    # the whole layer's workspace holds the 8-bit tokens and their scales, 256-byte padded, and the partial sums
    for m, n, k in ((1, 64, 100), (37, 5003, 4099), (128, 8192, 28672), (4096, 14336, 4096)):
        st, part = _size(lib.vq_q8_gemm_workspace_bytes, m, n, k)
        assert st == 0 and part % (4 * m * n) == 0
        pad = lambda b: (b + 255) // 256 * 256
        assert _size(lib.vq_q8_linear_workspace_bytes, m, n, k) == (0, pad(m * vq.q8_row_bytes(k)) + pad(4 * m) + pad(part))
    assert _size(lib.vq_q8_gemm_workspace_bytes, 128, 8192, 28672)[1] > 0
    f = lib.vq_q8_experts_workspace_bytes
    assert _size(f, 0, 2, 8, 64, 64) == (0, 0)
    st, n = _size(f, 100, 2, 8, 512, 300)
    assert st == 0 and n >= 200 * 300 * 4 + 200 * 512 * 4 + 100 * 512 + 200 * 384
    for bad in ((-1, 2, 8, 64, 64), (1, 0, 8, 64, 64), (1, 2, 0, 64, 64), (1, 2, 4097, 64, 64), (1, 2, 8, 0, 64),
                (1, 2, 8, 64, 65537), (1 << 29, 2, 8, 64, 64)):
        assert _size(f, *bad)[0] == vq.VQ_ERR_SHAPE
    assert f(1, 1, 1, 1, 1, None) == vq.VQ_ERR_NULL


def _refusals(f, good, cases, vq):
    for name, change, want in cases:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert f(*args) == getattr(vq, want), name


def test_quantize_refusals(vq):
    #        rows k  x  dtype ldx q  s  stream
    good = [4, 100, P, F16, 100, P, P, None]
    _refusals(vq.lib().vq_q8_quantize, good, [
        ("rows < 0", {0: -1}, "VQ_ERR_SHAPE"), ("k = 0", {1: 0, 4: 0}, "VQ_ERR_SHAPE"),
        ("k too long", {1: 65537, 4: 65537}, "VQ_ERR_SHAPE"), ("stride too short", {4: 99}, "VQ_ERR_SHAPE"),
        ("type", {3: BAD}, "VQ_ERR_UNSUPPORTED"), ("no x", {2: None}, "VQ_ERR_NULL"), ("no q", {5: None}, "VQ_ERR_NULL"),
        ("no s", {6: None}, "VQ_ERR_NULL"), ("x off", {2: P + 1}, "VQ_ERR_ALIGN"), ("q off", {5: P + 8}, "VQ_ERR_ALIGN"),
        ("s off", {6: P + 2}, "VQ_ERR_ALIGN"), ("fp32 x off", {2: P + 2, 3: F32}, "VQ_ERR_ALIGN"),
        ("no rows", {0: 0, 2: None, 5: None, 6: None}, "VQ_OK")], vq)


def test_gemm_refusals(vq):
    #        M  N   K   q  s  w  sw bias y dtype ws bytes stream
    good = [128, 8192, 28672, P, P, P, P, None, P, F16, P, 1 << 40, None]
    _refusals(vq.lib().vq_q8_gemm, good, [
        ("M < 0", {0: -1}, "VQ_ERR_SHAPE"), ("N < 0", {1: -1}, "VQ_ERR_SHAPE"), ("K = 0", {2: 0}, "VQ_ERR_SHAPE"),
        ("K too long", {2: 65537}, "VQ_ERR_SHAPE"), ("type", {9: BAD}, "VQ_ERR_UNSUPPORTED"),
        ("no q", {3: None}, "VQ_ERR_NULL"), ("no s", {4: None}, "VQ_ERR_NULL"), ("no w", {5: None}, "VQ_ERR_NULL"),
        ("no sw", {6: None}, "VQ_ERR_NULL"), ("no y", {8: None}, "VQ_ERR_NULL"), ("q off", {3: P + 8}, "VQ_ERR_ALIGN"),
        ("w off", {5: P + 4}, "VQ_ERR_ALIGN"), ("s off", {4: P + 2}, "VQ_ERR_ALIGN"), ("sw off", {6: P + 1}, "VQ_ERR_ALIGN"),
        ("bias off", {7: P + 1}, "VQ_ERR_ALIGN"), ("y off", {8: P + 1}, "VQ_ERR_ALIGN"),
        ("workspace off", {10: P + 128}, "VQ_ERR_ALIGN"), ("workspace short", {11: 1000}, "VQ_ERR_BUFFER_SIZE"),
        ("nothing", {0: 0, 3: None, 8: None}, "VQ_OK")], vq)


def test_linear_refusals(vq):
    #        M  N    K   x  dtype ldx  w  sw bias y dtype ws bytes stream
    good = [4, 300, 100, P, F16, 100, P, P, None, P, F16, P, 1 << 40, None]
    _refusals(vq.lib().vq_q8_linear, good, [
        ("M < 0", {0: -1}, "VQ_ERR_SHAPE"), ("K = 0", {2: 0}, "VQ_ERR_SHAPE"), ("stride", {5: 99}, "VQ_ERR_SHAPE"),
        ("x type", {4: BAD}, "VQ_ERR_UNSUPPORTED"), ("y type", {10: BAD}, "VQ_ERR_UNSUPPORTED"),
        ("no x", {3: None}, "VQ_ERR_NULL"), ("no w", {6: None}, "VQ_ERR_NULL"), ("no y", {9: None}, "VQ_ERR_NULL"),
        ("no workspace", {11: None}, "VQ_ERR_NULL"), ("short workspace", {12: 511}, "VQ_ERR_BUFFER_SIZE"),
        ("w off", {6: P + 8}, "VQ_ERR_ALIGN"), ("x off", {3: P + 1}, "VQ_ERR_ALIGN"), ("ws off", {11: P + 16}, "VQ_ERR_ALIGN"),
        ("no outputs", {1: 0, 3: None, 11: None}, "VQ_OK")], vq)


def test_expert_refusals(vq):
    lib = vq.lib()
    #        tokens top experts ids offsets rows pos stream
    _refusals(lib.vq_expert_plan, [4, 2, 8, P, P, P, P, None], [
        ("tokens", {0: -1}, "VQ_ERR_SHAPE"), ("top", {1: 0}, "VQ_ERR_SHAPE"), ("experts", {2: 0}, "VQ_ERR_SHAPE"),
        ("too many experts", {2: 4097}, "VQ_ERR_SHAPE"), ("too many pairs", {0: 1 << 29}, "VQ_ERR_SHAPE"),
        ("no ids", {3: None}, "VQ_ERR_NULL"), ("no offsets", {4: None}, "VQ_ERR_NULL"), ("no rows", {5: None}, "VQ_ERR_NULL"),
        ("no pos", {6: None}, "VQ_ERR_NULL"), ("ids off", {3: P + 2}, "VQ_ERR_ALIGN")], vq)
    #        experts max_rows tokens N K offsets rows q s w sw bias gated y dtype stream
    good = [8, 64, 32, 100, 200, P, P, P, P, P, P, None, 1, P, F32, None]
    _refusals(lib.vq_q8_gemm_grouped, good, [
        ("experts", {0: 0}, "VQ_ERR_SHAPE"), ("rows", {1: -1}, "VQ_ERR_SHAPE"), ("N", {3: -1}, "VQ_ERR_SHAPE"),
        ("K", {4: 0}, "VQ_ERR_SHAPE"), ("no tokens", {2: 0}, "VQ_ERR_SHAPE"),
        ("no gather and too few tokens", {6: None}, "VQ_ERR_SHAPE"), ("gated", {12: 2}, "VQ_ERR_UNSUPPORTED"),
        ("type", {14: BAD}, "VQ_ERR_UNSUPPORTED"), ("no offsets", {5: None}, "VQ_ERR_NULL"), ("no q", {7: None}, "VQ_ERR_NULL"),
        ("no w", {9: None}, "VQ_ERR_NULL"), ("no y", {13: None}, "VQ_ERR_NULL"), ("q off", {7: P + 8}, "VQ_ERR_ALIGN"),
        ("rows off", {6: P + 1}, "VQ_ERR_ALIGN"), ("y off", {13: P + 2}, "VQ_ERR_ALIGN"),
        ("nothing", {1: 0, 7: None}, "VQ_OK"), ("no outputs", {3: 0, 7: None}, "VQ_OK")], vq)
    #        tokens top N max_rows z pos p y dtype stream
    _refusals(lib.vq_expert_combine, [4, 2, 100, 8, P, P, P, P, F16, None], [
        ("tokens", {0: -1}, "VQ_ERR_SHAPE"), ("top", {1: 0}, "VQ_ERR_SHAPE"), ("N", {2: -1}, "VQ_ERR_SHAPE"),
        ("rows", {3: -1}, "VQ_ERR_SHAPE"), ("type", {8: BAD}, "VQ_ERR_UNSUPPORTED"), ("no z", {4: None}, "VQ_ERR_NULL"),
        ("no pos", {5: None}, "VQ_ERR_NULL"), ("no p", {6: None}, "VQ_ERR_NULL"), ("z off", {4: P + 2}, "VQ_ERR_ALIGN"),
        ("nothing", {0: 0, 5: None}, "VQ_OK")], vq)
    #        tokens top E D  I   x  dtype ldx ids p w_in s_in w_out s_out y dtype ws bytes stream
    good = [4, 2, 8, 64, 32, P, F16, 64, P, P, P, P, P, P, P, F16, P, 1 << 40, None]
    _refusals(lib.vq_q8_experts, good, [
        ("tokens", {0: -1}, "VQ_ERR_SHAPE"), ("top", {1: 0}, "VQ_ERR_SHAPE"), ("D", {3: 0}, "VQ_ERR_SHAPE"),
        ("I", {4: 65537}, "VQ_ERR_SHAPE"), ("stride", {7: 63}, "VQ_ERR_SHAPE"), ("x type", {6: BAD}, "VQ_ERR_UNSUPPORTED"),
        ("y type", {15: BAD}, "VQ_ERR_UNSUPPORTED"), ("no x", {5: None}, "VQ_ERR_NULL"), ("no p", {9: None}, "VQ_ERR_NULL"),
        ("no s_out", {13: None}, "VQ_ERR_NULL"), ("no workspace", {16: None}, "VQ_ERR_NULL"),
        ("short workspace", {17: 1000}, "VQ_ERR_BUFFER_SIZE"), ("w_in off", {10: P + 8}, "VQ_ERR_ALIGN"),
        ("ws off", {16: P + 64}, "VQ_ERR_ALIGN"), ("nothing", {0: 0, 5: None, 16: None}, "VQ_OK")], vq)


def test_block_norm_refusals(vq):
    base = dict(rows=4, dim=64, post=1, pre=1, z_dtype=F16, h_dtype=F16, w_dtype=F32, gate_dtype=F16, x_dtype=F16,
                gate_rows=1, eps=1e-6, w_offset=0, res_scale=1, gate_scale=1, ldz=64, ldh=64)
    order = ("z", "h", "post_w", "post_b", "pre_w", "pre_b", "gate", "r", "x", "q", "s")
    ptrs = dict.fromkeys(order, P)

    def call(desc=(), **ptr):
        d = vq.NormDesc(**(base | dict(desc)))
        return vq.lib().vq_block_norm(ctypes.byref(d), *((ptrs | ptr)[k] for k in order), None)

    assert vq.lib().vq_block_norm(None, *[P] * 11, None) == vq.VQ_ERR_NULL
    for desc in ({"rows": -1}, {"dim": 0}, {"dim": 65537, "ldz": 65537, "ldh": 65537}, {"ldz": 63}, {"ldh": 63},
                 {"gate_rows": 0}):
        assert call(desc) == vq.VQ_ERR_SHAPE, desc
    for desc in ({"post": 3}, {"pre": -1}, {"z_dtype": BAD}, {"h_dtype": BAD}, {"w_dtype": BAD}, {"gate_dtype": BAD},
                 {"x_dtype": BAD}, {"post": 0}, {"pre": 0}):
        assert call(desc) == vq.VQ_ERR_UNSUPPORTED, desc
    for ptr in ({"z": None}, {"q": None}, {"s": None}, {"r": None, "x": None, "q": None, "s": None}):
        assert call(**ptr) == vq.VQ_ERR_NULL, ptr
    for k in ("z", "h", "gate", "r", "x"):
        assert call(**{k: P + 1}) == vq.VQ_ERR_ALIGN, k
    for k in ("post_w", "post_b", "pre_w", "pre_b", "s"):
        assert call(**{k: P + 2}) == vq.VQ_ERR_ALIGN, k
    assert call(q=P + 8) == vq.VQ_ERR_ALIGN
    assert call({"rows": 0}, z=None, q=None) == vq.VQ_OK


def test_binding_refuses_host_tensors(vq):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        vq.q8_quantize(x)
    with pytest.raises(ValueError):
        vq.block_norm(x)
    with pytest.raises(ValueError):
        vq.expert_plan(torch.zeros((2, 2), dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        vq.Q8Linear(torch.zeros((4, 64), dtype=torch.int8), torch.ones(4))


def test_pad_on_the_host(vq):
    torch = pytest.importorskip("torch")
    w = torch.arange(-6, 6, dtype=torch.int8).reshape(2, 2, 3)
    p = vq.q8_pad(w)
    assert p.shape == (2, 2, 128) and torch.equal(p[..., :3], w) and not p[..., 3:].any()
    whole = torch.ones((2, 256), dtype=torch.int8)
    assert vq.q8_pad(whole).data_ptr() == whole.data_ptr()
