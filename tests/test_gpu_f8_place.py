"""Outputs of the 8-bit float layers in their input's place: the feed-forward layer's may be, a product's may not."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("m", [1, 7, 40, 300])
def test_in_place(m):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    g = torch.Generator(device="cuda").manual_seed(m)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    mlp, x = vq.F8MLP.from_weights(rnd(5000, 256) * 0.05, rnd(5000, 256) * 0.05, rnd(256, 5000) * 0.05), rnd(m, 256).bfloat16()
    want = mlp(x)
    ws = torch.empty(vq.f8_mlp_workspace_bytes(m, 256, 5000), dtype=torch.uint8, device="cuda")
    y = x.clone()
    assert vq.f8_mlp(y, mlp.w_in, mlp.s_in, mlp.w_out, mlp.s_out, 5000, ws, out=y) is y and torch.equal(y, want)
    lay = vq.F8Linear.from_weight(rnd(256, 256) * 0.05)
    ws = torch.empty(max(vq.f8_linear_workspace_bytes(m, 256, 256), 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(vq.VQError):
        vq.f8_linear(x, lay.w, lay.scale, None, ws, out=x)
