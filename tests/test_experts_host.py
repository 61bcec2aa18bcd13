"""Q8Experts and its weights on the host (no GPU)."""
import pytest

torch = pytest.importorskip("torch")


def test_layer_refuses_another_width(monkeypatch):
    """Columns and experts that the padding of rows hides: w_in for 100 columns beside w_out for 120."""
    import os

    import gemv_bit_unpack_amd as vq

    if not os.path.exists(vq.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    monkeypatch.setattr(vq.q8, "_device", lambda t, what: -1)
    i8, f32 = (lambda *s: torch.zeros(s, dtype=torch.int8)), (lambda *s: torch.zeros(s))
    for w_in in ((3, 32, 100), (3, 32, 127), (2, 32, 120), (3, 30, 120)):
        with pytest.raises(ValueError, match="w_in must be"):
            vq.Q8Experts(i8(*w_in), f32(3, 32), i8(3, 120, 16), f32(3, 120))
    for w_in in ((3, 32, 120), (3, 32, 128)):  # as it is, and padded already
        layer = vq.Q8Experts(i8(*w_in), f32(3, 32), i8(3, 120, 16), f32(3, 120))
        assert (layer.experts, layer.features, layer.inner) == (3, 120, 16)
