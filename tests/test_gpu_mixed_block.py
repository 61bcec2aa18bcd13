"""The example block runs all of it together: norms -> 8-bit projection -> codebook projection -> norms -> experts.

Against the same block in fp32 on the decoded weights it differs by the 8-bit steps of the tokens and hidden rows and by
the bf16 stores.  A row of unit-normal values spans about +-3.3 over 1024 columns, so an 8-bit step is 6.6 / 254 and its
rounding 0.0075 of the row's spread; the hidden rows' product of two normals spans about three times as far: 0.02.  bf16
adds 0.002 a store.  The residual takes one such error through the projections, the experts' output both: 0.02 and 0.05
leave room for twice that.  A router's near-tie may go the other way in one of them: rows whose choice differs are left out.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("tokens", [1, 3, 40, 300])
def test_block(tokens):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gemv_bit_unpack_amd.examples.mixed_block import MixedBlock

    block = MixedBlock()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    mlp, r = (torch.randn((tokens, 1024), generator=g, device="cuda").bfloat16() for _ in range(2))
    chosen, route = [], block.route

    def noted(x):
        ids, p = route(x)
        chosen.append(ids.sort(dim=1).values)
        return ids, p

    block.route = noted
    (y, r1), (y64, r64) = block.step(mlp, r), block.step_fp32(mlp, r)
    rel = lambda a, b: float((a.float() - b).norm() / b.norm())
    assert rel(r1, r64) <= 0.02
    same = (chosen[0] == chosen[1]).all(dim=1)
    assert int(same.sum()) >= 0.9 * tokens - 1
    if bool(same.any()):
        assert rel(y[same], y64[same]) <= 0.05
    # two steps in a row, from the outputs of the first
    y2, r2 = block.step(y, r1)
    assert bool(torch.isfinite(y2).all()) and bool(torch.isfinite(r2).all())
