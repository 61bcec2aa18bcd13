"""The grouped product in every tile size that its rule takes (by the rows of a group on average, and by whether the CUs
hold all tiles at once): within the product's derived bound, and the bits of the dense product, group by group.
"""
import numpy as np
import pytest

import q8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("e,avg,n,k,gated", [
    (3, 4, 100, 200, True), (5, 3, 333, 65, True),                       # 32-row tiles
    (4, 30, 200, 300, True), (7, 96, 70, 129, True),                     # 64
    (4, 97, 260, 140, True), (6, 150, 300, 200, True), (3, 400, 130, 70, True),   # 256
    (9, 48, 300, 257, False),                                            # 32
    (4, 60, 400, 300, False), (5, 190, 129, 130, False),                 # 128: few tiles
    (40, 64, 900, 130, False), (30, 190, 700, 200, False), (24, 100, 1500, 500, False),   # 64: more than 256 tiles of 128
    (4, 193, 500, 260, False), (2, 700, 257, 128, False),                # 256
])
def test_ways(e, avg, n, k, gated):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as vq

    print("grouped", e, avg, n, k, gated, flush=True)
    g = np.random.default_rng([e, avg, n, k])
    m = e * avg
    cuts = np.sort(g.integers(0, m + 1, e - 1))          # ragged groups, some of them empty
    if e > 3:
        cuts[1] = cuts[0]
    off = np.concatenate([[0], cuts, [m]]).astype(np.int32)
    rows = g.permutation(m).astype(np.int32)
    wn = 2 * n if gated else n
    w = g.integers(-127, 128, (e, wn, k)).astype(np.int8)
    sw = g.uniform(1e-3, 2e-3, (e, wn)).astype(np.float32)
    bias = (g.standard_normal((e, wn)) * 0.2).astype(np.float16)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    x = torch.from_numpy(g.standard_normal((m, k)).astype(np.float32)).cuda()
    q, s = vq.q8_quantize(x)
    wd, swd = vq.q8_pad(cu(w)), cu(sw)
    qn, sn = q[:, :k].cpu().numpy(), s.cpu().numpy()
    for b in (None, bias):
        y = vq.q8_gemm_grouped(cu(off), cu(rows), q, s, wd, swd, None if b is None else cu(b), k, m, gated=gated)
        for ex in range(e):
            lo, hi = off[ex], off[ex + 1]
            if lo == hi:
                continue
            f = q8ref.gated if gated else q8ref.product
            ref, bound = f(qn[rows[lo:hi]], sn[rows[lo:hi]], w[ex], sw[ex], None if b is None else b[ex])
            q8ref.check(y[lo:hi], ref, bound, "f32")
            if not gated:
                r = torch.from_numpy(rows[lo:hi].astype(np.int64)).cuda()
                dense = vq.q8_gemm(q[r], s[r], wd[ex], swd[ex], None if b is None else cu(b[ex]), k, y_dtype=torch.float32)
                assert torch.equal(y[lo:hi], dense)
