"""The 8-bit float products in every way that the rule takes (tests/test_f8_ways_host.py holds the list to it), on whole numbers
with scales that are powers of two: sums are exact in every order and operand form, so dense outputs have to be equal bit for
bit, and gated ones within the gate's own error, of 16-bit types too."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import f8ways  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E = 2.0 ** -24


@pytest.fixture(scope="module")
def vq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_bit_unpack_amd as g

    g.lib()
    return g


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _gen(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) & 0x7FFFFFFF)


def _silu(g):
    return g / (1 + torch.exp(-g))


@pytest.mark.parametrize("m,n,k,gated", f8ways.SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_exact(vq, m, n, k, gated, dt):
    g = _gen(m, n, k)
    x = f8ways.tokens(g, m, k, DT[dt])
    w, sw, w64 = f8ways.weights(g, n, k, 2 if gated else 1, f8ways.unit_shift(k) if gated else 0)
    w = vq.f8_pad(w)
    y64 = x.double() @ w64.t().contiguous()
    del w64
    # steps of 64 * 2^-4 (dense; as many more powers of two down with the gate): 24 bits hold the sums
    assert float(y64.abs().max()) < 64 * 2.0 ** (f8ways.unit_shift(k) if gated else 0) * 2 ** 19
    if gated:
        a, u = _silu(y64[:, :n]), y64[:, n:]
        # the gate: exp to 2 ulp, one addition, one division, two products
        y64, bound = a * u, 8 * E * (a * u).abs() + 1e-36 * u.abs()
    q, s = vq.f8_quantize(x)
    assert torch.equal(q[:, :k].double() * s.double().t().repeat_interleave(128, 1)[:, :k], x.double())
    for out in ("f32", "bf16", "f16"):
        print("ways", m, n, k, gated, dt, out, sorted(f8ways.ways(vq.lib(), m, n, k, gated)), flush=True)
        got = [vq.f8_linear(x, w, sw, None, _ws(vq.f8_linear_workspace_bytes(m, n, k, gated)), gated=gated, y_dtype=DT[out]),
               vq.f8_gemm(q, s, w, sw, None, k, gated=gated, ws=_ws(vq.f8_gemm_workspace_bytes(m, n, k, gated)),
                          y_dtype=DT[out]),
               vq.f8_gemm(q, s, w, sw, None, k, gated=gated, y_dtype=DT[out])]
        torch.cuda.synchronize()
        want = y64.float().to(DT[out])  # fp32 holds the dense sums
        for i, y in enumerate(got):
            if not gated:
                assert torch.equal(y, want), i
                continue
            keep = want.isfinite()  # past the largest fp16 value
            half = torch.finfo(DT[out]).eps / 2
            off = (y.double() - y64).abs() - bound - half * (y64.abs() + bound) - torch.finfo(DT[out]).smallest_normal * half
            assert bool((off[keep] <= 0).all()) and torch.equal(y[~keep], want[~keep]), (i, float(off[keep].max()))


@pytest.mark.parametrize("m,d,i,hidden", f8ways.LAYERS)
@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f32", "bf16")])
def test_hidden_rows(vq, m, d, i, hidden, dt, out):
    """The hidden rows themselves, by an output projection that picks one column for each output: equal, but for values so near
    the border of two e4m3 steps that the gate's error takes them over it (8 E of a step of 2^-4: 1.5e-5 of them)."""
    g = _gen(m, d, i)
    x = f8ways.tokens(g, m, d, DT[dt])
    w, sw, w64 = f8ways.weights(g, i, d, 2, f8ways.unit_shift(d))
    y64 = x.double() @ w64.t().contiguous()
    h = (_silu(y64[:, :i]) * y64[:, i:]).float()
    blocks = -(-i // 128)
    padded = torch.nn.functional.pad(h, (0, blocks * 128 - i)).view(m, blocks, 128)
    s = padded.abs().amax(2, keepdim=True) / torch.full((1,), 448.0, device="cuda")  # by a tensor: a true division
    v = torch.where(s > 0, padded / s, torch.zeros_like(padded)).clamp(-448, 448).to(f8ways.E4).float()
    v, s = v.view(m, -1)[:, :i], s.expand(-1, -1, 128).reshape(m, -1)[:, :i]
    cols = torch.cat((torch.arange(blocks, device="cuda") * 128, torch.tensor([i - 1], device="cuda"),
                      torch.randint(0, i, (d,), generator=g, device="cuda")))[:d]
    cols = torch.minimum(cols, torch.tensor(i - 1, device="cuda"))
    pick = torch.zeros((d, i), device="cuda")
    pick[torch.arange(d, device="cuda"), cols] = 1.0
    print("hidden", m, d, i, hidden, dt, out, flush=True)
    y = vq.F8MLP(w, sw, pick.to(f8ways.E4), torch.ones((-(-d // 128), blocks), device="cuda"))(x, DT[out])
    torch.cuda.synchronize()
    want, step = (v * s)[:, cols], (v.abs() * 2.0 ** -3).clamp(min=2.0 ** -9)[:, cols] * s[:, cols]
    half = torch.finfo(DT[out]).eps / 2
    off = (y.double() - want.double()).abs()
    # the same value of 8 bits: its scale is off by the largest value's gate (8 E) and a rounding on either side; the row here
    # is rounded to fp32 first, and value times scale is once more on either side, there to the output's type
    near = off <= (12 * E + half) * want.abs()
    assert bool((off <= step * 1.01 + half * want.abs()).all())
    assert int((~near).sum()) <= 4 + 1e-4 * near.numel(), int((~near).sum())
