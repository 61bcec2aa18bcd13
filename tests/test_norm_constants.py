"""block_norm's constants are read at every call: a tensor given for one counts with the value it has then."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def seen(monkeypatch):
    """The descriptors that block_norm hands to the library, whose launch is replaced."""
    import os

    import gemv_bit_unpack_amd as vq

    if not os.path.exists(vq.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    real, got = vq.lib(), []

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def vq_block_norm(self, desc, *args):
            d = ctypes.cast(desc, ctypes.POINTER(vq.NormDesc)).contents
            got.append({n: getattr(d, n) for n in ("eps", "w_offset", "res_scale", "gate_scale")})
            return 0

    monkeypatch.setattr(vq.q8, "lib", lambda: Lib())
    monkeypatch.setattr(vq.q8, "_device", lambda t, what: -1)
    monkeypatch.setattr(vq.q8, "_stream", lambda dev: 0)
    return vq, got


@pytest.mark.parametrize("name,field", [("gate_scale", "gate_scale"), ("res_scale", "res_scale"), ("eps", "eps"),
                                        ("weight_offset", "w_offset")])
@pytest.mark.parametrize("make", [lambda: torch.tensor(0.5), lambda: torch.nn.Parameter(torch.tensor(0.5))])
def test_a_tensor_updated_in_place(seen, name, field, make):
    vq, got = seen
    z, scale = torch.zeros((2, 64)), make()
    for value in (0.5, 0.25, 0.125):
        with torch.no_grad():
            scale.fill_(value)
        vq.block_norm(z, z, **{name: scale})
        assert got[-1][field] == value


def test_the_sign_of_zero_does_not_depend_on_the_call_before(seen):
    import math

    vq, got = seen
    z = torch.zeros((3, 64))
    for order in ((0.0, -0.0), (-0.0, 0.0)):
        vq.q8._norm_desc.cache_clear()
        signs = set()
        for v in order:
            vq.block_norm(z, z, gate_scale=v)
            signs.add(math.copysign(1.0, got[-1]["gate_scale"]))
        assert signs == {1.0}


def test_no_tensor_is_kept(seen):
    import gc
    import weakref

    vq, _ = seen
    scale = torch.tensor(0.5)
    gone = weakref.ref(scale)
    vq.block_norm(torch.zeros((2, 64)), gate_scale=scale)
    del scale
    gc.collect()
    assert gone() is None
