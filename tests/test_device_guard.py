"""Every call launches with its tensors' device current, whichever was before, and gives that one back.

The default stream of every device has the handle 0: with another device current, a launch on it would go there.  On the
host, device 1 is stood in for by tensors of the CPU and a library that notes the current device.
"""
import pytest

torch = pytest.importorskip("torch")

LAUNCHES = ("vq_dequant", "vq_gemv", "vq_gemv_ws", "vq_gemv_noalloc", "vq_gemm", "vq_gemm_ws", "vq_gemv_ws_rht",
            "vq_gemm_ws_rht", "vq_svq_dequant", "vq_svq_gemv", "vq_svq_gemm", "vq_rht", "vq_assign", "vq_q8_quantize",
            "vq_q8_gemm", "vq_q8_linear", "vq_expert_plan", "vq_q8_gemm_grouped", "vq_expert_combine", "vq_q8_experts",
            "vq_block_norm")


class _Devices:
    """The current device, as torch's two switches of it see it."""

    def __init__(self):
        self.now = 0

    def exchange(self, dev):
        was, self.now = self.now, dev if dev >= 0 else self.now
        return was


class _On1(torch.Tensor):
    def get_device(self):
        return 1


@pytest.fixture
def rig(monkeypatch):
    import ctypes
    import os

    import gemv_bit_unpack_amd as vq

    if not os.path.exists(vq.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    real, cur, seen, result = vq.lib(), _Devices(), [], [0]

    class Lib:
        def __getattr__(self, name):
            if name not in LAUNCHES:
                return getattr(real, name)

            def launch(*args):
                seen.append((name, cur.now))
                return result[0]

            launch.__name__ = name
            return launch

    monkeypatch.setattr(torch._C, "_cuda_exchangeDevice", cur.exchange, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_maybeExchangeDevice", cur.exchange, raising=False)
    for mod in (vq, vq.q8):
        monkeypatch.setattr(mod, "lib", lambda: Lib())
    monkeypatch.setattr(vq, "_dev_ptr", lambda t, what, dtypes=None: None if t is None else ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(vq, "_stream_ptr", lambda device: None)
    monkeypatch.setattr(vq.q8, "_device", lambda t, what: 1)
    monkeypatch.setattr(vq.q8, "_stream", lambda dev: 0)
    monkeypatch.setattr(vq.q8, "_ptr", lambda t, *a: None if t is None else t.data_ptr())
    return vq, cur, seen, result


def _calls(vq):
    on1 = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt).as_subclass(_On1)
    f32 = lambda *s: on1(*s, dt=torch.float32)
    i8, i32 = lambda *s: on1(*s, dt=torch.int8), lambda *s: on1(*s, dt=torch.int32)
    u8 = lambda *s: on1(*s, dt=torch.uint8)
    d, ld = vq.make_desc(16, 64, 8, 8, 0), vq.svq_desc(16, 64)
    vqa, sva = (d, u8(4096), on1(256, 8), None, on1(16)), (ld, u8(4096), on1(4, 4), on1(4), on1(16))
    x = on1(2, 64)
    for name in ("gemv", "gemv_noalloc", "gemm"):
        yield lambda name=name: getattr(vq, name)(*vqa, None, x)
    for name in ("gemv_ws", "gemm_ws"):
        yield lambda name=name: getattr(vq, name)(*vqa, None, x, None)
    for name in ("gemv_ws_rht", "gemm_ws_rht"):
        yield lambda name=name: getattr(vq, name)(*vqa, None, x, u8(8), None)
    for name in ("svq_gemv", "svq_gemm"):
        yield lambda name=name: getattr(vq, name)(*sva, None, x)
    yield lambda: vq.dequant(*vqa)
    yield lambda: vq.svq_dequant(*sva)
    yield lambda: vq.rht(x, u8(8))
    yield lambda: vq.assign(d, on1(16, 64), on1(256, 8))
    q, s = i8(2, 128), f32(2)
    yield lambda: vq.q8_quantize(x)
    yield lambda: vq.q8_gemm(q, s, i8(16, 128), f32(16), None, 64)
    yield lambda: vq.q8_linear(x, i8(16, 128), f32(16), None, None)
    yield lambda: vq.expert_plan(i32(2, 2), 4)
    yield lambda: vq.q8_gemm_grouped(i32(5), i32(4), q, s, i8(4, 16, 128), f32(4, 16), None, 64, 4)
    yield lambda: vq.expert_combine(f32(4, 16), i32(2, 2), f32(2, 2))
    ex = (i8(4, 32, 128), f32(4, 32), i8(4, 64, 128), f32(4, 64))
    yield lambda: vq.q8_experts(x, i32(2, 2), f32(2, 2), *ex, 16, None)
    yield lambda: vq.block_norm(x)
    lin = vq.Q8Linear(i8(16, 128), f32(16))
    yield lambda: lin(on1(2, 128))
    yield lambda: lin.forward_q8(q, s)
    lay = vq.Q8Experts(i8(4, 32, 128), f32(4, 32), i8(4, 128, 16), f32(4, 128))
    yield lambda: lay(on1(2, 128), i32(2, 2), f32(2, 2))


def test_every_launch_finds_its_device(rig):
    vq, cur, seen, _ = rig
    for before in (0, 1):
        cur.now = before
        for call in _calls(vq):
            n = len(seen)
            call()
            assert seen[n:] and all(dev == 1 for _, dev in seen[n:]), seen[n:]
            assert cur.now == before, seen[n:]
    assert {name for name, _ in seen} == set(LAUNCHES)


def test_given_back_after_a_refusal(rig):
    vq, cur, seen, result = rig
    result[0] = vq.VQ_ERR_SHAPE
    for call in _calls(vq):
        with pytest.raises(vq.VQError) as e:
            call()
        assert cur.now == 0 and str(e.value).startswith(seen[-1][0])


@pytest.mark.gpu
def test_on_the_gpu():
    """The only device there is stays current, on a refusal too."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    dev = torch.cuda.current_device()
    _, y = vq.block_norm(torch.ones((2, 64), device="cuda"))
    assert float((y - 1).abs().max()) < 1e-6
    with pytest.raises(vq.VQError):
        vq.q8_quantize(torch.zeros((1, 65537), device="cuda"))
    assert torch.cuda.current_device() == dev
