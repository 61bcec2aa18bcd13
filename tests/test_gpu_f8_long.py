"""vq_f8_quantize on more rows of weights than 65535 blocks."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_many_rows_of_weights():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    rows = 65536 * 128 + 77
    x = torch.randn((rows, 2), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    q, s = vq.f8_quantize(x, 128)
    assert s.shape == (65537, 1)
    for lo, hi in ((0, 256), (65534 * 128, rows)):  # blocks on both sides of the bound, as they are by themselves
        part, scale = vq.f8_quantize(x[lo:hi], 128)
        assert torch.equal(s[lo // 128:-(-hi // 128)], scale) and torch.equal(q[lo:hi].view(torch.uint8), part.view(torch.uint8))
    big = torch.nn.functional.pad(x.float().abs(), (0, 0, 0, 128 - 77)).view(-1, 256).amax(1)
    assert torch.equal(s.flatten(), big / torch.full((1,), 448.0, device="cuda"))  # by a tensor: a true division
