"""The operators of a block with layers in 8-bit floating point and of its heads' positions, as measured cases.

Four operators that stand between the codebook-quantized layers of a block:

  linear   y = x W^T (+ bias) with W in 8-bit floats (e4m3) and one fp32 scale for each 128 x 128 block of it; x is cut
           to 8-bit floats inside the call, with one fp32 scale for each 128 values of a token.
  mlp      y = W_out (silu(g) * u), (g, u) = W_in x: the same product twice; the gated activation is cut to 8-bit floats
           again in between.  The gate's and the up projection's rows have blocks of their own.
  rotate   rotary positions of queries and keys: pairs of a head's values turned by position * frequency, in the half
           layout (j, j + dim / 2) or interleaved (2 j, 2 j + 1), on the whole head or a part, with frequencies scaled for
           long contexts.
  heads    the same with a norm over each head's values first.

8-bit tokens: s = max|x| / 448 per block and x / s, both in fp32; q is the quotient rounded to the nearest e4m3 value,
ties to even (a zero block: s = q = 0).  Blocks at the ends are short.

``run`` computes the plain form in elementary fp32 torch operations (angles in fp64), or, with ``own``, calls the package.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BLOCK = 128
TOP = 448.0  # the largest e4m3 value


def linear(name, m, n, k, dtype, out=None, bias=False):
    return {"name": name, "kind": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "out": out or dtype, "bias": bias}


def mlp(name, m, d, i, dtype):
    return {"name": name, "kind": "mlp", "m": m, "d": d, "i": i, "dtype": dtype}


def heads(name, batch, t, hq, hk, d, dtype, norm="none", rot=None, start=0, interleaved=False, scaling="none", far=4096,
          decode=False, bias=False):
    return {"name": name, "kind": "rotate" if norm == "none" else "heads", "batch": batch, "t": t, "hq": hq, "hk": hk,
            "d": d, "dtype": dtype, "norm": norm, "rot": rot or d, "start": start, "interleaved": interleaved,
            "scaling": scaling, "far": far, "decode": decode, "bias": bias}


def listed():
    return [
        # one token through a 4096 x 4096 attention projection: the smallest product, launch latency counts
        linear("linear_4k_m1", 1, 4096, 4096, "f16"),
        # one token through the 70B-class up projection: 235 MB of weights, memory bound
        linear("linear_70b_up_m1", 1, 28672, 8192, "bf16"),
        # a batch of 37 sequences in decode: odd sizes, short blocks at both ends, a bias, fp32 outputs
        linear("linear_odd_m37", 37, 5003, 4099, "bf16", out="f32", bias=True),
        # 128 sequences in decode through the 70B-class down projection: between memory and matrix bound
        linear("linear_70b_down_m128", 128, 8192, 28672, "bf16"),
        # a prompt of 4096 tokens through the 8B-class up projection: matrix bound
        linear("linear_8b_up_m4096", 4096, 14336, 4096, "bf16"),
        # one token through the 8B-class MLP: 176 MB of weights
        mlp("mlp_8b_m1", 1, 4096, 14336, "bf16"),
        # 77 sequences in decode through a small MLP of odd sizes
        mlp("mlp_odd_m77", 77, 2056, 5001, "f16"),
        # a prompt of 2048 tokens through the 8B-class MLP: matrix bound
        mlp("mlp_8b_m2048", 2048, 4096, 14336, "bf16"),
        # 16 sequences in decode, each at its own far position, contexts stretched 16 times: launch latency counts
        heads("rotate_m16", 16, 1, 32, 8, 128, "bf16", scaling="yarn", far=1 << 20, decode=True),
        # two prompts of 4096 tokens, half of each head rotated in the interleaved layout: memory bound
        heads("rotate_2x4096", 2, 4096, 64, 8, 128, "f16", rot=64, start=64, interleaved=True, scaling="linear"),
        # one token of a model with norms on its queries and keys: the smallest pass
        heads("heads_m1", 1, 1, 64, 8, 128, "bf16", norm="rms", scaling="bands", far=1 << 17, decode=True),
        # a prompt of 8192 tokens of the same model: memory bound
        heads("heads_m8192", 1, 8192, 64, 8, 128, "bf16", norm="rms"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("linear", "linear", "mlp", "heads", "heads"))
    while True:
        if kind == "linear":
            dtype = rng.choice(("f16", "bf16", "f32"))
            c = linear("", log_int(rng, 1, 4096), log_int(rng, 64, 28672), log_int(rng, 64, 28672), dtype,
                       rng.choice((dtype, "f32")), rng.random() < 0.5)
            fits = c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096
        elif kind == "mlp":
            c = mlp("", log_int(rng, 1, 4096), log_int(rng, 64, 8192), log_int(rng, 64, 28672), rng.choice(("f16", "bf16")))
            fits = c["m"] * c["d"] * c["i"] <= 2048 * 4096 * 14336 and c["d"] * c["i"] <= 4096 * 14336
        else:
            hk = log_int(rng, 1, 32)
            d = rng.choice((32, 64, 80, 96, 112, 128, 128, 192, 256, 2 * rng.randint(8, 160)))
            rot = rng.choice((d, d, d // 2 // 2 * 2, 2 * rng.randint(1, d // 2)))
            decode = rng.random() < 0.4
            c = heads("", log_int(rng, 1, 64), 1 if decode else log_int(rng, 1, 8192), hk * rng.choice((1, 2, 4, 8)), hk, d,
                      rng.choice(("f16", "bf16", "f32")), rng.choice(("none", "rms", "rms", "layer")), rot,
                      rng.choice((0, d - rot)), rng.random() < 0.5, rng.choice(("none", "linear", "ntk", "yarn", "bands")),
                      log_int(rng, 4096, 1 << 20), decode, rng.random() < 0.3)
            size = c["batch"] * c["t"] * (c["hq"] + 2 * hk) * d * (2 if c["dtype"] == "f32" else 1)
            fits = size <= 8192 * 80 * 128
        if fits:
            del c["name"]
            return c


def frequencies(case):
    """Radians per position of each pair (Python floats) and the factor on the rotated values.  Stretching a context of
    `old` positions s times:
      linear  every angle at 1 / s of its speed           ntk   the base grows so that the slowest pair does
      yarn    a ramp between the two ends: pairs that turn more than 32 times in `old` positions keep their speed, those
              that turn less than once get 1 / s of it; rotated values times 0.1 ln s + 1
      bands   wavelengths below old / 4 keep theirs, above old / 1 get 1 / s, in between by the turns in `old` positions
    """
    rot, base, s, old, kind = case["rot"], 500000.0, 16.0, 8192, case["scaling"]
    if kind == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if kind == "linear":
        return [v / s for v in f], 1.0
    if kind == "yarn":
        at = lambda turns: rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = lambda j: min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        return [v / s * ramp(j) + v * (1 - ramp(j)) for j, v in enumerate(f)], 0.1 * math.log(s) + 1.0
    if kind == "bands":
        mix = lambda v: min(max((old * v / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0)
        return [mix(v) * v + (1 - mix(v)) * v / s for v in f], 1.0
    return f, 1.0


def activations(g, m, d, dtype, spread=1.0):
    """Tokens as a block meets them: unit spread, and about one channel in 200 with values ten times as large."""
    x = torch.randn((m, d), generator=g, device="cuda") * spread
    loud = torch.rand((d,), generator=g, device="cuda") < 0.005
    return (x * torch.where(loud, 10.0, 1.0)).to(DT[dtype])


def weights8(g, n, k):
    """e4m3 weights [n, k] and the scales of their 128 x 128 blocks: a spread near 0.02 that differs between blocks."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = (torch.randn((n, k), generator=g, device="cuda") * 100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    return w, (torch.rand((nb, kb), generator=g, device="cuda") + 0.5) * (0.02 / 100.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if own:
        import gemv_bit_unpack_amd as vq
    if case["kind"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        w, s = weights8(g, n, k)
        bias = (torch.randn((n,), generator=g, device="cuda") * 0.1).half() if case["bias"] else None
        st |= {"x": activations(g, m, k, case["dtype"]), "w": w, "s": s, "bias": bias}
        if own:
            st["layer"] = vq.F8Linear(w, s, bias)
    elif case["kind"] == "mlp":
        m, d, i = case["m"], case["d"], case["i"]
        gate, up, out = weights8(g, i, d), weights8(g, i, d), weights8(g, d, i)
        st |= {"x": activations(g, m, d, case["dtype"]), "w_in": torch.cat((gate[0].view(torch.uint8), up[0].view(torch.uint8))),
               "s_in": torch.cat((gate[1], up[1])), "w_out": out[0], "s_out": out[1]}
        st["w_in"] = st["w_in"].view(torch.float8_e4m3fn)
        if own:
            st["layer"] = vq.F8MLP(st["w_in"], st["s_in"], st["w_out"], st["s_out"])
    else:
        b, t, hq, hk, d = (case[x] for x in ("batch", "t", "hq", "hk", "d"))
        # what the projection in front of the heads wrote: queries, keys and values side by side
        st["qkv"] = activations(g, b * t, (hq + 2 * hk) * d, case["dtype"]).reshape(b, t, (hq + 2 * hk) * d)
        if case["decode"]:  # every sequence at a position of its own
            pos = torch.randint(0, case["far"], (b, 1), generator=g, device="cuda")
        else:  # prompts, or chunks of long ones, from some position on
            pos = torch.randint(0, max(case["far"] - t, 1), (b, 1), generator=g, device="cuda") + torch.arange(t, device="cuda")
        st["positions"] = pos
        vec = lambda scale, shift: torch.randn((d,), generator=g, device="cuda") * scale + shift
        normed = case["norm"] != "none"
        for x in ("q", "k"):
            st[x + "_w"] = vec(0.1, 1.0) if normed else None
            st[x + "_b"] = vec(0.1, 0.0) if normed and case["bias"] else None
        if own:
            scaling = {"none": None, "linear": {"kind": "linear", "factor": 16.0}, "ntk": {"kind": "ntk", "factor": 16.0},
                       "yarn": {"kind": "yarn", "factor": 16.0, "length": 8192},
                       "bands": {"kind": "bands", "factor": 16.0, "length": 8192, "low": 1.0, "high": 4.0}}[case["scaling"]]
            st["rotary"] = vq.Rotary(case["rot"], base=500000.0, start=case["start"], interleaved=case["interleaved"],
                                     scaling=scaling, device="cuda")
        else:
            f, st["scale"] = frequencies(case)
            st["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    return st


def split_heads(st):
    """The queries [batch, t, hq, d] and keys [batch, t, hk, d], views of the projection's output."""
    c = st["case"]
    b, t, hq, hk, d = (c[x] for x in ("batch", "t", "hq", "hk", "d"))
    return st["qkv"][..., :hq * d].view(b, t, hq, d), st["qkv"][..., hq * d:(hq + hk) * d].view(b, t, hk, d)


# ------------------------------------------------------------------ plain forms (fp32)

def to8(x):
    """Rows of fp32 values as the values that their 8-bit floats stand for."""
    m, k = x.shape
    kb = -(-k // BLOCK)
    b = torch.zeros((m, kb * BLOCK), device=x.device)
    b[:, :k] = x
    b = b.view(m, kb, BLOCK)
    s = b.abs().amax(dim=2, keepdim=True) / torch.full((1,), TOP, device=x.device)  # by a tensor: a true division
    q = torch.where(s > 0, (b / s).clamp(-TOP, TOP), torch.zeros_like(b)).to(torch.float8_e4m3fn).float()
    return (q * s).view(m, kb * BLOCK)[:, :k]


def spread_blocks(s, n, k):
    return s.repeat_interleave(BLOCK, dim=0)[:n].repeat_interleave(BLOCK, dim=1)[:, :k]


def plain_product(x, w, s):
    n, k = w.shape
    return torch.matmul(to8(x), (w.float() * spread_blocks(s, n, k)).t())


def plain_heads(st):
    c = st["case"]
    angle = st["positions"].double().unsqueeze(-1) * st["freqs"]
    cos, sin = (f(angle).unsqueeze(2) * st["scale"] for f in (torch.cos, torch.sin))
    cos, sin = cos.float(), sin.float()
    out = []
    for x, w, b in zip(split_heads(st), (st["q_w"], st["k_w"]), (st["q_b"], st["k_b"])):
        x = x.float()
        if c["norm"] == "layer":
            x = x - x.mean(dim=-1, keepdim=True)
        if c["norm"] != "none":
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w
            x = x if b is None else x + b
        at, rot = c["start"], c["rot"]
        part = x[..., at:at + rot]
        if c["interleaved"]:
            u, v = part[..., 0::2], part[..., 1::2]
            turned = torch.stack((u * cos - v * sin, u * sin + v * cos), dim=-1).flatten(-2)
        else:
            u, v = part[..., :rot // 2], part[..., rot // 2:]
            turned = torch.cat((u * cos - v * sin, u * sin + v * cos), dim=-1)
        out.append(torch.cat((x[..., :at], turned, x[..., at + rot:]), dim=-1).to(DT[c["dtype"]]))
    return tuple(out)


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        import gemv_bit_unpack_amd as vq

        if kind == "linear":
            return st["layer"].forward(st["x"], y_dtype=DT[case["out"]])
        if kind == "mlp":
            return st["layer"].forward(st["x"])
        q, k = split_heads(st)
        return vq.rotate_heads(q, k, st["positions"], st["rotary"], norm=case["norm"], q_weight=st["q_w"], q_bias=st["q_b"],
                               k_weight=st["k_w"], k_bias=st["k_b"], eps=EPS)

    if kind in ("rotate", "heads"):
        return plain_heads(st)
    if kind == "linear":
        y = plain_product(st["x"].float(), st["w"], st["s"])
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return y.to(DT[case["out"]])
    gu = plain_product(st["x"].float(), st["w_in"][:case["i"]], st["s_in"][:st["s_in"].shape[0] // 2])
    u = plain_product(st["x"].float(), st["w_in"][case["i"]:], st["s_in"][st["s_in"].shape[0] // 2:])
    return plain_product(gu * torch.sigmoid(gu) * u, st["w_out"], st["s_out"]).to(DT[case["dtype"]])


# ------------------------------------------------------------------ the definition in 64 bits

def exact_tokens(x):
    """Tokens as the values that their 8-bit floats stand for, by arithmetic: e4m3 has steps of 2^(e - 3) from 2^e on, and
    of 2^-9 below 2^-6.  The definition holds the scale and the quotient in fp32 (a value next to the middle of two steps
    would otherwise go either way)."""
    cols = []
    for part in x.split(BLOCK, dim=1):
        s = (part.abs().max(dim=1).values / TOP).float().double()[:, None]
        v = (part / torch.where(s > 0, s, torch.ones_like(s))).float().double()
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        cols.append((torch.round(v / step) * step).clamp(-TOP, TOP) * s)
    return torch.cat(cols, dim=1)


def exact_product(x, w, s):
    x = exact_tokens(x)
    out = []
    for r, rows in enumerate(w.split(BLOCK * 32, dim=0)):  # channels in parts, to bound the 64-bit copy of the weights
        scale = s[r * 32:r * 32 + 32].double()
        wide = rows.double()
        for b in range(scale.shape[0]):
            for c in range(scale.shape[1]):
                wide[b * BLOCK:(b + 1) * BLOCK, c * BLOCK:(c + 1) * BLOCK] *= scale[b, c]
        out.append(x @ wide.t().contiguous())
    return torch.cat(out, dim=1)


def exact_heads(st):
    c = st["case"]
    at, rot, d = c["start"], c["rot"], c["d"]
    f, scale = frequencies(c)
    turn = torch.polar(torch.full((rot // 2,), scale, dtype=torch.float64, device="cuda").expand(*st["positions"].shape, -1),
                       st["positions"].double()[..., None] * torch.tensor(f, dtype=torch.float64, device="cuda"))[:, :, None]
    first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1) + at
    second = first + (1 if c["interleaved"] else rot // 2)
    out = []
    for x, w, b in zip(split_heads(st), (st["q_w"], st["k_w"]), (st["q_b"], st["k_b"])):
        y = x.double()
        if c["norm"] != "none":
            centre = y.sum(dim=3, keepdim=True) / d if c["norm"] == "layer" else 0.0
            y = (y - centre) / torch.sqrt(((y - centre) ** 2).sum(dim=3, keepdim=True) / d + EPS) * w.double()
            y = y + (0.0 if b is None else b.double())
        else:
            y = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["kind"] in ("rotate", "heads"):
        return exact_heads(st)
    x = st["x"].double()
    if case["kind"] == "linear":
        y = exact_product(x, st["w"], st["s"])
        return y if st["bias"] is None else y + st["bias"].double()
    i, half = case["i"], st["s_in"].shape[0] // 2
    g, u = (exact_product(x, st["w_in"][a:a + i], st["s_in"][b:b + half]) for a, b in ((0, 0), (i, half)))
    return exact_product(g / (1.0 + torch.exp(-g)) * u, st["w_out"], st["s_out"])


def work(case):
    size = lambda name: 4 if name == "f32" else 2
    blocks = lambda n, k: 4 * (-(-n // BLOCK)) * (-(-k // BLOCK))
    if case["kind"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k + blocks(n, k) + (2 * n if case["bias"] else 0) + m * k * size(case["dtype"])
                + m * n * size(case["out"]), "flops": 2 * m * n * k}
    if case["kind"] == "mlp":
        m, d, i = case["m"], case["d"], case["i"]
        return {"bytes": 3 * d * i + 3 * blocks(d, i) + 2 * m * d * size(case["dtype"]), "flops": 6 * m * d * i}
    b, t, hq, hk, d = (case[x] for x in ("batch", "t", "hq", "hk", "d"))
    vecs = 0 if case["norm"] == "none" else 4 if case["bias"] else 2
    return {"bytes": 2 * b * t * (hq + hk) * d * size(case["dtype"]) + 8 * b * t + 4 * vecs * d + 4 * case["rot"],
            "flops": b * t * (hq + hk) * ((0 if vecs == 0 else 4 * d) + 3 * case["rot"])}
