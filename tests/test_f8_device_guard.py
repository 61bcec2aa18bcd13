"""Every call of the 8-bit float layers and of rotate_heads launches with its tensors' device current, whichever was before,
and gives that one back, on a refusal too.  On the host, device 1 is stood in for by tensors of the CPU and a library that
notes the current device."""
import pytest

torch = pytest.importorskip("torch")

LAUNCHES = ("vq_f8_quantize", "vq_f8_gemm", "vq_f8_linear", "vq_f8_mlp", "vq_rotate_heads")


class _On1(torch.Tensor):
    def get_device(self):
        return 1


@pytest.fixture
def rig(monkeypatch):
    import os

    import gemv_bit_unpack_amd as vq

    if not os.path.exists(vq.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    real, now, seen, result = vq.lib(), [0], [], [0]

    class Lib:
        def __getattr__(self, name):
            if name not in LAUNCHES:
                return getattr(real, name)

            def launch(*args):
                seen.append((name, now[0]))
                return result[0]

            launch.__name__ = name
            return launch

    def exchange(dev):
        was, now[0] = now[0], dev if dev >= 0 else now[0]
        return was

    monkeypatch.setattr(torch._C, "_cuda_exchangeDevice", exchange, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_maybeExchangeDevice", exchange, raising=False)
    for mod in (vq, vq.q8, vq.f8, vq.heads):
        monkeypatch.setattr(mod, "lib", lambda: Lib())
    for mod in (vq.q8, vq.f8, vq.heads):
        monkeypatch.setattr(mod, "_device", lambda t, what: 1)
        monkeypatch.setattr(mod, "_stream", lambda dev: 0)
        monkeypatch.setattr(mod, "_ptr", lambda t, *a: None if t is None else t.data_ptr())
    return vq, now, seen, result


def _calls(vq):
    on1 = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt).as_subclass(_On1)
    f32, e4 = (lambda *s: on1(*s, dt=torch.float32)), (lambda *s: on1(*s, dt=torch.float8_e4m3fn))
    x, q, s = on1(2, 64), e4(2, 128), f32(1, 2)
    yield lambda: vq.f8_quantize(x)
    yield lambda: vq.f8_gemm(q, s, e4(16, 128), f32(1, 1), None, 64)
    yield lambda: vq.f8_linear(x, e4(16, 128), f32(1, 1), None, None)
    yield lambda: vq.f8_mlp(x, e4(32, 128), f32(2, 1), e4(64, 128), f32(1, 1), 16, None)
    lin = vq.F8Linear(e4(16, 128), f32(1, 1))
    yield lambda: lin(on1(2, 128))
    yield lambda: lin.forward_f8(q, s)
    mlp = vq.F8MLP(e4(32, 128), f32(2, 1), e4(128, 16), f32(1, 1))
    yield lambda: mlp(on1(2, 128))
    rotary = vq.Rotary(8, device="cpu")
    rotary._dev = 1
    yield lambda: vq.rotate_heads(on1(3, 2, 8), on1(3, 1, 8), on1(3, dt=torch.int64), rotary)


def test_every_launch_finds_its_device(rig):
    vq, now, seen, _ = rig
    for before in (0, 1):
        now[0] = before
        for call in _calls(vq):
            n = len(seen)
            call()
            assert seen[n:] and all(dev == 1 for _, dev in seen[n:]), seen[n:]
            assert now[0] == before
    assert {name for name, _ in seen} == set(LAUNCHES)


def test_given_back_after_a_refusal(rig):
    vq, now, seen, result = rig
    result[0] = vq.VQ_ERR_SHAPE
    for call in _calls(vq):
        with pytest.raises(vq.VQError) as e:
            call()
        assert now[0] == 0 and str(e.value).startswith(seen[-1][0])


def test_other_devices_are_refused(rig, monkeypatch):
    """Tensors of two devices in one call."""
    vq, *_ = rig
    monkeypatch.undo()
    on1 = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt).as_subclass(_On1)
    rotary = vq.Rotary(8, device="cpu")
    with pytest.raises(ValueError, match="device"):
        vq.rotate_heads(on1(3, 2, 8), torch.zeros((3, 1, 8), dtype=torch.float16), on1(3, dt=torch.int64), rotary)
    with pytest.raises(ValueError, match="device"):
        vq.rotate_heads(on1(3, 2, 8), None, on1(3, dt=torch.int64), rotary)
    with pytest.raises(ValueError, match="device"):
        vq.f8_gemm(on1(2, 128, dt=torch.float8_e4m3fn), torch.zeros((1, 2)), torch.zeros((16, 128), dtype=torch.float8_e4m3fn),
                   torch.zeros((1, 1)), None, 64)
