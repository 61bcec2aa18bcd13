"""The example block runs all of it together: norms -> 8-bit float projection -> norms and rotation of the heads -> attention
-> codebook projection -> norms -> gated feed-forward layer in 8-bit floats.

Against the same block in fp64 on the decoded weights it differs by the tokens' 8-bit rounding and the bf16 stores.  An e4m3
value is off by at most 2^-4 of itself, evenly spread over half steps of 2^-4 to 2^-5: 0.026 (rms).  The weights are the
decoded ones on both sides, so each product takes 0.026 from its tokens.  Queries and keys enter the scores, whose spread of 1
they move by 0.026 * sqrt 2 each way, and values the weighted sum: 0.026 + 0.037 through the attention at most, halved again
in the residual, which is the sum of three parts of one size.  The feed-forward layer takes its tokens' 0.026 twice (gate and
up), its hidden rows' 0.026, and the residual's own error: under 0.1 together.  A single token attends to itself alone.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("tokens", [1, 3, 40, 300])
def test_block(tokens):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gemv_bit_unpack_amd.examples.f8_block import F8Block

    block = F8Block()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    mlp, r = (torch.randn((tokens, 1024), generator=g, device="cuda").bfloat16() for _ in range(2))
    pos = torch.arange(tokens, device="cuda") + 70000
    (y, r1), (y64, r64) = block.step(mlp, r, pos), block.step_fp64(mlp, r, pos)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(r1, r64) <= 0.05 and rel(y, y64) <= 0.1, (rel(r1, r64), rel(y, y64))
    # two steps in a row, and a graph of one replayed, from the outputs of the first
    y2, r2 = block.step(y, r1, pos)
    assert bool(torch.isfinite(y2).all()) and bool(torch.isfinite(r2).all())


def test_positions_matter():
    """Another position of a later token changes what it attends to, and only the difference of positions does."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gemv_bit_unpack_amd.examples.f8_block import F8Block

    block = F8Block()
    g = torch.Generator(device="cuda").manual_seed(0)
    mlp, r = (torch.randn((16, 1024), generator=g, device="cuda").bfloat16() for _ in range(2))
    pos = torch.arange(16, device="cuda")
    y = block.step(mlp, r, pos)[1].double()
    far = block.step(mlp, r, pos + 1000000)[1].double()
    other = block.step(mlp, r, pos * 50)[1].double()
    rel = lambda a, b: float((a - b).norm() / b.norm())
    # bf16 queries and keys are rounded differently at other positions: 2^-9 of each, in scores of spread 1
    assert rel(far, y) < 0.01 < rel(other, y)
