"""The dense product of few rows on both sides of every bound between the streamed form and the tiles: within its derived
bound, and each row the bits that it has alone in a product of many (another form)."""
import numpy as np
import pytest

import q8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("m", [1, 8, 9, 16, 17, 32, 33, 48, 49, 64, 65])
@pytest.mark.parametrize("n,k", [
    (1000, 900), (1000, 1025), (1030, 2048), (3001, 2049), (1500, 4096), (1500, 4097), (1024, 8192), (1023, 7169),   # 16 rows a group, one round
    (4097, 1024), (4200, 1025), (4608, 300),                                         # 16 rows a group, two rounds
    (4609, 1024), (5003, 4096), (6000, 4097), (7200, 8192), (8192, 1000), (8192, 1025), (7169, 8193),    # 32, one round
    (8193, 2048), (9001, 2049), (12287, 300),                                         # 32, two rounds
    (12288, 300), (12300, 2048)])                                                      # 64
def test_both_sides(m, n, k):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    g = torch.Generator(device="cuda").manual_seed(m * 1000003 + n * 31 + k)
    w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand((n,), generator=g, device="cuda") * 1e-3 + 5e-4
    q, s = vq.q8_quantize(torch.randn((m, k), generator=g, device="cuda"))
    wd = vq.q8_pad(w)
    nb = vq.q8_gemm_workspace_bytes(m, n, k)
    y = torch.full((m + 2, n), 7.0, device="cuda")
    vq.q8_gemm(q, s, wd, sw, None, k, ws=torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None, out=y[1:m + 1])
    assert bool((y[0] == 7).all()) and bool((y[m + 1] == 7).all())
    many = vq.q8_gemm(q.repeat(-(-300 // m), 1), s.repeat(-(-300 // m)), wd, sw, None, k, y_dtype=torch.float32)
    assert torch.equal(y[1:m + 1], many[:m])
    cols = [0, 1, 15, 16, 31, 32, 63, 64, n // 2, n - 17, n - 2, n - 1]
    ref, bound = q8ref.product(q[:, :k].cpu().numpy(), s.cpu().numpy(), w[cols].cpu().numpy(), sw[cols].cpu().numpy())
    q8ref.check(y[1:m + 1][:, cols], ref, bound, "f32")
