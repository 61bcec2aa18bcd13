"""The 8-bit layers take every view of their tokens, as VQLinear does: transposed, expanded, overlapping and reversed
batches give the bits of a contiguous copy."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layers():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    g = np.random.default_rng(21)
    w = lambda *s: torch.from_numpy(g.integers(-127, 128, s).astype(np.int8)).cuda()
    sc = lambda *s: torch.from_numpy(g.uniform(1e-3, 3e-3, s).astype(np.float32)).cuda()
    lin = vq.Q8Linear(w(40, 100), sc(40))
    exp = vq.Q8Experts(w(3, 64, 100), sc(3, 64), w(3, 100, 32), sc(3, 100))

    def experts(x):
        m = x[..., 0].numel()
        r = torch.arange(m, device="cuda", dtype=torch.int32)
        return exp(x, torch.stack([r % 3, (r + 1) % 3], dim=1).contiguous(), torch.full((m, 2), 0.5, device="cuda"))

    return {"linear": lin, "experts": experts}


def _views():
    base = torch.randn((6, 5, 100), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    flat = base.reshape(-1)
    return {
        "expanded": base[0, :1].expand(7, 100),
        "expanded in 3-d": base[:, :1].expand(6, 4, 100),
        "one row expanded once": base[0, :1].expand(1, 100),
        "overlapping": flat.as_strided((9, 100), (30, 1)),
        "transposed": torch.randn((100, 8), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half().t(),
        "one value for all columns": base[0, :, :1].expand(5, 100),
        "every other row": base.reshape(30, 100)[::2],
        "batch transposed": base.transpose(0, 1),
    }


@pytest.mark.parametrize("layer", ["linear", "experts"])
def test_views(layers, layer):
    call = layers[layer]
    for name, x in _views().items():
        got, want = call(x), call(x.contiguous().clone())
        assert got.shape == want.shape and torch.equal(got, want), name
