"""rotate_heads with positions that are views: expanded, rows of a wider tensor, a column of it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_views():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    g = torch.Generator(device="cuda").manual_seed(1)
    rotary = vq.Rotary(64)
    q, k = (torch.randn((3, 5, h, 64), generator=g, device="cuda").bfloat16() for h in (4, 2))
    wide = torch.randint(0, 1 << 20, (6, 9), generator=g, device="cuda")
    for dt in (torch.int64, torch.int32):
        pos = wide.to(dt)
        for view in (pos[0, :5].expand(3, 5), pos[::2, 2:7], pos[:3, 4:]):
            got, want = vq.rotate_heads(q, k, view, rotary), vq.rotate_heads(q, k, view.contiguous(), rotary)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
        one = pos[:3, 7:8]
        got, want = (vq.rotate_heads(q[:, :1], k[:, :1], p, rotary) for p in (one, one.contiguous()))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
