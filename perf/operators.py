"""The operators of an 8-bit transformer block beside the codebook layers, as measured cases.

Three operators that a block with some layers kept in 8 bits runs next to its codebook-quantized ones:

  linear   y = x W^T (+ bias) with W in 8-bit integers and one fp32 scale per output channel; x is cut to 8-bit
           integers with one fp32 scale per token inside the call.  Cases with ``norm`` begin at the block's entry:
           the residual add and both norms write the 8-bit tokens that the product reads.
  experts  y[t] = sum_j p[t, j] W_out[e] (silu(g) * u), (g, u) = W_in[e] x[t], e = ids[t, j]: the same 8-bit product
           grouped by expert with ragged group sizes, the gated activation cut to 8 bits again in between.
  norm     r = res_scale * h + gate_scale * gate * N_post(z), x = N_pre(r): the norms after one block and before the
           next, fused with the gate and the residual add.

8-bit tokens: s = max|x| / 127 per row and x / s, both in fp32; q is the quotient rounded to nearest even, within +-127
(a zero row: s = q = 0).

``run`` computes the plain form in elementary fp32 torch operations, or, with ``own``, calls the package.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def linear(name, m, n, k, dtype, out=None, bias=False, norm=False):
    return {"name": name, "kind": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "out": out or dtype, "bias": bias,
            "norm": norm}


def experts(name, t, e, top, d, i, dtype):
    return {"name": name, "kind": "experts", "t": t, "e": e, "top": top, "d": d, "i": i, "dtype": dtype}


def norm(name, m, d, z, r, x, post, pre, gate, gate_rows=1, bias=False):
    return {"name": name, "kind": "norm", "m": m, "d": d, "z": z, "r": r, "x": x, "post": post, "pre": pre,
            "gate": gate, "gate_rows": gate_rows, "bias": bias}


def listed():
    return [
        # one token through a 4096 x 4096 attention projection: the smallest product, launch latency counts
        linear("linear_4k_m1", 1, 4096, 4096, "f16"),
        # one token through the 70B-class up projection: 235 MB of weights, memory bound
        linear("linear_70b_up_m1", 1, 28672, 8192, "bf16"),
        # a block's entry for a batch of 37 sequences in decode: both norms, the residual add, then a projection of odd sizes
        linear("linear_entry_odd_m37", 37, 5003, 4099, "bf16", bias=True, norm=True),
        # 128 sequences in decode through the 70B-class down projection: between memory and matrix bound
        linear("linear_70b_down_m128", 128, 8192, 28672, "bf16"),
        # a prompt of 4096 tokens through the 8B-class up projection: matrix bound
        linear("linear_8b_up_m4096", 4096, 14336, 4096, "bf16"),
        # one token through 2 of 8 experts with the 8B-class MLP's sizes: six launches over 352 MB of weights
        experts("experts_8x8b_t1", 1, 8, 2, 4096, 14336, "bf16"),
        # 333 tokens over 64 small experts: short ragged groups, some empty
        experts("experts_64_t333", 333, 64, 4, 2048, 1024, "bf16"),
        # a prompt of 4096 tokens through 2 of 8 experts with the 8B-class MLP's sizes: matrix bound
        experts("experts_8x8b_t4096", 4096, 8, 2, 4096, 14336, "bf16"),
        # one token of a 4096-wide model between two blocks: pre-norm only, launch latency counts
        norm("norm_4k_m1", 1, 4096, "f16", "f16", "f16", "none", "rms", "none"),
        # 64 sequences in decode of an 8192-wide model: norms on both sides and a learned gate for each channel
        norm("norm_8k_m64", 64, 8192, "bf16", "bf16", "bf16", "rms", "rms", "channel"),
        # odd sizes: centred norms with biases, an fp32 residual stream and one gate row for every 111 tokens
        norm("norm_odd_m333", 333, 5003, "f16", "f32", "f16", "layer", "layer", "rows", 111, True),
        # a prompt of 8192 tokens of an 8192-wide model: memory bound
        norm("norm_8k_m8192", 8192, 8192, "bf16", "bf16", "bf16", "rms", "rms", "channel"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("linear", "linear", "experts", "norm"))
    while True:
        if kind == "linear":
            c = linear("", log_int(rng, 1, 4096), log_int(rng, 64, 28672), log_int(rng, 64, 28672),
                       rng.choice(("f16", "bf16")), rng.choice(("f16", "bf16", "f32")), rng.random() < 0.5)
            c["norm"] = c["k"] <= 16384 and rng.random() < 0.3
            if c["norm"]:
                c["dtype"] = c["out"] = "bf16"
            fits = c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096
        elif kind == "experts":
            e = log_int(rng, 2, 128)
            c = experts("", log_int(rng, 1, 4096), e, rng.randint(1, min(8, e)), log_int(rng, 128, 4096),
                        log_int(rng, 128, 14336), rng.choice(("f16", "bf16")))
            fits = e * c["d"] * c["i"] <= 8 * 4096 * 14336 and c["t"] * c["top"] * c["d"] * c["i"] <= 8192 * 4096 * 14336
        else:
            z = rng.choice(("f16", "bf16", "f32"))
            m = log_int(rng, 1, 8192)
            c = norm("", m, log_int(rng, 64, 16384), z, rng.choice((z, "f32")), z, rng.choice(("none", "rms", "layer")),
                     rng.choice(("rms", "layer")), rng.choice(("none", "channel", "rows")), rng.randint(1, m),
                     rng.random() < 0.5)
            fits = m * c["d"] <= 4096 * 8192
        if fits:
            del c["name"]
            return c


def activations(g, m, d, dtype, spread=1.0):
    """Tokens as a block meets them: unit spread, and about one channel in 200 with values ten times as large."""
    x = torch.randn((m, d), generator=g, device="cuda") * spread
    loud = torch.rand((d,), generator=g, device="cuda") < 0.005
    return (x * torch.where(loud, 10.0, 1.0)).to(DT[dtype])


def weights8(g, n, k):
    """8-bit weights [n, k] and their channels' scales: a weight spread near 0.02."""
    w = (torch.randn((n, k), generator=g, device="cuda") * 32.0).round_().clamp_(-127, 127).to(torch.int8)
    return w, (torch.rand((n,), generator=g, device="cuda") + 0.5) * (0.02 / 32.0)


def prepare_norm(g, m, d, z, r, post, pre, gate, gate_rows, bias):
    dev = {"device": "cuda", "generator": g}
    vec = lambda scale, shift: torch.randn((d,), **dev) * scale + shift
    rows = 1 if gate == "channel" else -(-m // gate_rows)
    return {
        "z": activations(g, m, d, z, 0.5), "h": activations(g, m, d, r, 2.0), "post": post, "pre": pre,
        "post_w": None if post == "none" else vec(0.05, 0.5), "pre_w": vec(0.1, 1.0),
        "post_b": vec(0.1, 0.0) if bias and post != "none" else None, "pre_b": vec(0.1, 0.0) if bias else None,
        "gate": None if gate == "none" else (torch.rand((rows, d), **dev) * 2 - 1).to(DT[z]),
        "gate_rows": m if gate == "channel" else gate_rows, "res_scale": 1.0, "gate_scale": 0.7,
    }


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["kind"] == "norm":
        st |= prepare_norm(g, case["m"], case["d"], case["z"], case["r"], case["post"], case["pre"], case["gate"],
                           case["gate_rows"], case["bias"])
    elif case["kind"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        w, s = weights8(g, n, k)
        bias = (torch.randn((n,), generator=g, device="cuda") * 0.1).half() if case["bias"] else None
        if case["norm"]:
            st |= prepare_norm(g, m, k, case["dtype"], case["dtype"], "rms", "rms", "none", 1, False)
        else:
            st["x"] = activations(g, m, k, case["dtype"])
        st |= {"w": w, "s": s, "bias": bias}
        if own:
            import gemv_bit_unpack_amd as vq

            st["layer"] = vq.Q8Linear(w, s, bias)
    else:
        t, e, d, i = case["t"], case["e"], case["d"], case["i"]
        w_in, s_in, w_out, s_out = [], [], [], []
        for _ in range(e):
            a, b = weights8(g, 2 * i, d)
            w_in.append(a), s_in.append(b)
            a, b = weights8(g, d, i)
            w_out.append(a), s_out.append(b)
        st |= {"w_in": torch.stack(w_in), "s_in": torch.stack(s_in), "w_out": torch.stack(w_out),
               "s_out": torch.stack(s_out), "x": activations(g, t, d, case["dtype"])}
        del w_in, w_out
        # router scores: some experts are liked more than others
        score = torch.randn((t, e), generator=g, device="cuda") + 0.7 * torch.randn((e,), generator=g, device="cuda")
        top, ids = score.topk(case["top"], dim=1)
        st |= {"ids": ids.to(torch.int32), "p": torch.softmax(top, dim=1)}
        if own:
            import gemv_bit_unpack_amd as vq

            st["layer"] = vq.Q8Experts(st["w_in"], st["s_in"], st["w_out"], st["s_out"])
    return st


# ------------------------------------------------------------------ plain forms (fp32)

def normed(a, kind, w, b):
    if kind == "none":
        return a
    if kind == "layer":
        a = a - a.mean(dim=1, keepdim=True)
    a = a * torch.rsqrt((a * a).mean(dim=1, keepdim=True) + EPS) * w
    return a if b is None else a + b


def plain_norm(st):
    u = normed(st["z"].float(), st["post"], st["post_w"], st["post_b"])
    if st["gate"] is not None:
        m = u.shape[0]
        u = u * st["gate"].float().repeat_interleave(st["gate_rows"], dim=0)[:m]
    r = st["res_scale"] * st["h"].float() + st["gate_scale"] * u
    return r, normed(r, st["pre"], st["pre_w"], st["pre_b"])


def to8(x):
    """Rows of fp32 values as 8-bit integers (held in fp32) and their scales."""
    big = x.abs().amax(dim=1, keepdim=True)
    s = big / torch.full_like(big, 127.0)  # by a tensor: a true division (by a number torch multiplies by 1 / 127)
    return torch.where(s > 0, (x / s).round().clamp(-127, 127), torch.zeros_like(x)), s


def plain_product(q, s, w, sw):
    return torch.matmul(q, w.float().t()) * s * sw


def plain_experts(st):
    x, ids, p = st["x"].float(), st["ids"], st["p"]
    i = st["w_out"].shape[2]
    q, s = to8(x)
    y = torch.zeros_like(x)
    for e in range(st["w_in"].shape[0]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if tok.numel() == 0:
            continue
        gu = plain_product(q[tok], s[tok], st["w_in"][e], st["s_in"][e])
        hq, hs = to8(gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:])
        y[tok] += plain_product(hq, hs, st["w_out"][e], st["s_out"][e]) * p[tok, slot].unsqueeze(1)
    return y


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        import gemv_bit_unpack_amd as vq

        if "z" in st:
            kw = dict(post=st["post"], post_weight=st["post_w"], post_bias=st["post_b"], pre=st["pre"],
                      pre_weight=st["pre_w"], pre_bias=st["pre_b"], gate=st["gate"], gate_rows=st["gate_rows"],
                      res_scale=st["res_scale"], gate_scale=st["gate_scale"], eps=EPS)
        if case["kind"] == "norm":
            return vq.block_norm(st["z"], st["h"], x_dtype=DT[case["x"]], **kw)
        if case["kind"] == "experts":
            return st["layer"].forward(st["x"], st["ids"], st["p"])
        if case["norm"]:
            r, q, s = vq.block_norm(st["z"], st["h"], q8=True, **kw)
            return r, st["layer"].forward_q8(q, s, y_dtype=DT[case["out"]])
        return st["layer"].forward(st["x"], y_dtype=DT[case["out"]])

    if case["kind"] == "norm":
        r, x = plain_norm(st)
        return r.to(DT[case["r"]]), x.to(DT[case["x"]])
    if case["kind"] == "experts":
        return plain_experts(st).to(DT[case["dtype"]])
    r, x = plain_norm(st) if case["norm"] else (None, st["x"].float())
    q, s = to8(x)
    y = plain_product(q, s, st["w"], st["s"])
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = y.to(DT[case["out"]])
    return (r.to(DT[case["dtype"]]), y) if case["norm"] else y


# ------------------------------------------------------------------ the definition in 64 bits

def exact_norm(st):
    def one(a, kind, w, b):
        if kind == "none":
            return a
        centre = a.sum(dim=1) / a.shape[1] if kind == "layer" else torch.zeros_like(a[:, 0])
        c = a - centre[:, None]
        a = c / torch.sqrt((c ** 2).sum(dim=1) / a.shape[1] + EPS)[:, None] * w.double()
        return a if b is None else a + b.double()

    u = one(st["z"].double(), st["post"], st["post_w"], st["post_b"])
    if st["gate"] is not None:
        row = torch.arange(u.shape[0], device=u.device) // st["gate_rows"]
        u = st["gate"].double()[row] * u
    r = st["h"].double() * st["res_scale"] + u * st["gate_scale"]
    return r, one(r, st["pre"], st["pre_w"], st["pre_b"])


def exact_tokens(x):
    """8-bit tokens times their scales.  The definition holds the scale and the quotient in fp32 (a value of half the
    row's largest lies on a tie, which the scale's rounding would otherwise break either way)."""
    s = (x.abs().max(dim=1).values / 127.0).float().double()[:, None]
    q = torch.round((x / torch.where(s > 0, s, torch.ones_like(s))).float().double()).clamp(-127, 127)
    return q * s


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["kind"] == "norm":
        return exact_norm(st)
    if case["kind"] == "linear":
        r, x = exact_norm(st) if case["norm"] else (None, st["x"].double())
        x = exact_tokens(x)
        cols = []
        for at in range(0, case["n"], 4096):  # channels in blocks, to bound the 64-bit copy of the weights
            cols.append(x @ (st["w"][at:at + 4096].double() * st["s"][at:at + 4096].double()[:, None]).t().contiguous())
        y = torch.cat(cols, dim=1)
        if st["bias"] is not None:
            y = y + st["bias"].double()
        return (r, y) if case["norm"] else y
    x = exact_tokens(st["x"].double())
    y = torch.zeros_like(x)
    i = case["i"]
    for e in range(case["e"]):
        share = torch.where(st["ids"] == e, st["p"].double(), torch.zeros((), dtype=torch.float64, device=x.device)).sum(dim=1)
        rows = torch.nonzero((st["ids"] == e).any(dim=1)).flatten()
        if rows.numel() == 0:
            continue
        gu = x[rows] @ (st["w_in"][e].double() * st["s_in"][e].double()[:, None]).t().contiguous()
        h = exact_tokens(gu[:, :i] / (1.0 + torch.exp(-gu[:, :i])) * gu[:, i:])
        y[rows] += share[rows][:, None] * (h @ (st["w_out"][e].double() * st["s_out"][e].double()[:, None]).t().contiguous())
    return y


def work(case):
    size = lambda name: 4 if name == "f32" else 2
    if case["kind"] == "norm":
        m, d = case["m"], case["d"]
        rows = {"none": 0, "channel": 1, "rows": -(-m // case["gate_rows"])}[case["gate"]]
        vecs = (case["pre"] != "none") + (case["post"] != "none")
        vecs *= 1 + bool(case["bias"])
        by = m * d * (size(case["z"]) + 2 * size(case["r"]) + size(case["x"])) + rows * d * size(case["z"]) + 4 * vecs * d
        return {"bytes": by, "flops": 12 * m * d}
    if case["kind"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        tokens = m * k * size(case["dtype"]) * (3 if case["norm"] else 1) + (8 * k if case["norm"] else 0)
        return {"bytes": n * k + 4 * n + (2 * n if case["bias"] else 0) + tokens + m * n * size(case["out"]),
                "flops": 2 * m * n * k}
    t, e, top, d, i = (case[x] for x in ("t", "e", "top", "d", "i"))
    hit = e * (1.0 - (1.0 - top / e) ** t)  # experts that some token chose, were they all alike
    return {"bytes": int(hit * (3 * i * d + 4 * (2 * i + d))) + 2 * t * d * size(case["dtype"]) + 8 * t * top,
            "flops": 6 * t * top * d * i}
