"""A call of several launches refuses a size that one of them has no grid for before the first is made.  No GPU is
needed: a call that launched would fail with another error here.  Pointers are made-up addresses."""
import pytest

P = 1 << 20


@pytest.fixture(scope="module")
def vq():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    return g


# tokens, top, D, I
@pytest.mark.parametrize("size", [
    (100_000_000, 8, 16, 16),      # the hidden rows' pass: four rows to a workgroup
    (80_000_000, 1, 16, 16),       # the tokens' pass
    (4_000_000, 1, 32768, 513),    # the join: a thread for each four outputs
])
def test_experts(vq, size):
    tokens, top, d, i = size
    call = lambda t: vq.lib().vq_q8_experts(t, top, 8, d, i, P, 0, d, P, P, P, P, P, P, P, 0, P, 1 << 62, None)
    assert call(tokens) == vq.VQ_ERR_SHAPE
