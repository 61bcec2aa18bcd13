"""A decoder block whose dense layers are in 8-bit floats with block scales, step by step through the library:

    python -m gemv_bit_unpack_amd.examples.f8_block [--tokens 1] [--steps 8]

    r, x    = block_norm(mlp, r, pre)                    residual add, norm before
    qkv     = F8Linear(x)                                8-bit float projection
    q, k    = rotate_heads(q, k, positions, rotary)      norms of the heads, rotary positions, in place
    a       = causal attention in plain torch            (the library has none)
    o       = VQLinear(a)                                codebook-quantized projection
    r, x    = block_norm(o, r, pre)                      the same between the halves of the block
    mlp     = F8MLP(x)                                   gated feed-forward layer

Weights are random.  Prints the time of a step and how far it is from the same block in fp64 on the decoded weights.
"""
from __future__ import annotations

import argparse

import numpy as np


def decoded(w, s, n, k):
    """The values of e4m3 weights [n, ..] with the scales of their 128 x 128 blocks, in fp64."""
    full = s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return w[:n, :k].double() * full


class F8Block:
    def __init__(self, dim=1024, heads=8, kv_heads=2, inner=1792, device="cuda", seed=0):
        import torch

        import gemv_bit_unpack_amd as vq

        self.vq, self.torch, self.dim, self.heads, self.kv_heads, self.inner = vq, torch, dim, heads, kv_heads, inner
        self.head = dim // heads
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)
        self.norms = [0.1 * rnd(dim) + 1 for _ in range(2)]
        self.q_norm, self.k_norm = (0.1 * rnd(self.head) + 1 for _ in range(2))
        self.qkv = vq.F8Linear.from_weight(rnd((heads + 2 * kv_heads) * self.head, dim) / dim ** 0.5)
        self.rotary = vq.Rotary(self.head, 500000.0, device=device,
                                scaling={"kind": "bands", "factor": 8.0, "length": 8192, "low": 1.0, "high": 4.0})
        hr = np.random.default_rng(seed)
        desc = vq.make_desc(dim, dim, 8, 16, 8)
        self.out = vq.VQLinear.from_indices(
            desc, hr.integers(0, 1 << 16, (dim, dim // 8), dtype=np.uint32), hr.integers(0, 256, (dim, dim // 8), dtype=np.uint32),
            (rnd(1 << 16, 8) / dim ** 0.5).half(), (0.2 * rnd(256, 8) / dim ** 0.5).half(),
            (torch.rand((dim,), generator=g, device=device) + 0.5).half(), device=device)
        self.mlp = vq.F8MLP.from_weights(rnd(inner, dim) / dim ** 0.5, rnd(inner, dim) / dim ** 0.5, rnd(dim, inner) / inner ** 0.5)

    def split(self, qkv):
        """Views of the projection's output: queries, keys and values [tokens, heads, head]."""
        t, d, cut = qkv.shape[0], self.head, self.heads * self.head
        kv = self.kv_heads * d
        return (qkv[:, :cut].view(t, self.heads, d), qkv[:, cut:cut + kv].view(t, self.kv_heads, d),
                qkv[:, cut + kv:].view(t, self.kv_heads, d))

    def attention(self, q, k, v):
        torch = self.torch
        t, share = q.shape[0], self.heads // self.kv_heads
        q, k, v = (x.to(torch.float64 if x.dtype is torch.float64 else torch.float32).transpose(0, 1) for x in (q, k, v))
        k, v = (x.repeat_interleave(share, 0).contiguous() for x in (k, v))
        score = q.contiguous() @ k.transpose(1, 2).contiguous() / self.head ** 0.5
        score = score.masked_fill(torch.ones((t, t), dtype=torch.bool, device=q.device).triu(1), -float("inf"))
        return (torch.softmax(score, -1) @ v).transpose(0, 1).reshape(t, self.dim)

    def step(self, mlp, r, positions):
        """(mlp output, residual) of the block before -> the same of this one; both [tokens, dim] bf16."""
        vq, n = self.vq, self.norms
        r, x = vq.block_norm(mlp, r, pre="rms", pre_weight=n[0])
        q, k, v = self.split(self.qkv(x))
        vq.rotate_heads(q, k, positions, self.rotary, norm="rms", q_weight=self.q_norm, k_weight=self.k_norm, q_out=q, k_out=k)
        o = self.out(self.attention(q, k, v).bfloat16())
        r, x = vq.block_norm(o, r, pre="rms", pre_weight=n[1])
        return self.mlp(x), r

    def step_fp64(self, mlp, r, positions):
        """The same block in fp64 on the decoded weights, nothing rounded in between."""
        torch, vq, n = self.torch, self.vq, self.norms
        rms = lambda a, w: a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6) * w.double()
        l, m, d = self.qkv, self.mlp, self.out
        r = r.double() + mlp.double()
        q, k, v = self.split(rms(r, n[0]) @ decoded(l.w, l.scale, l.out_features, self.dim).t().contiguous())
        angle = positions.double()[:, None] * self.rotary.freqs * (2 * np.pi)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        half = self.head // 2

        def rotated(x, w):
            x = rms(x, w)
            z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
            return torch.cat((z.real, z.imag), -1)

        o = self.attention(rotated(q, self.q_norm), rotated(k, self.k_norm), v)
        r = r + o @ vq.dequant(d.desc, d.packed, d.cb1, d.cb2, d.scale).double().t().contiguous()
        x = rms(r, n[1])
        blocks = m.s_in.shape[0] // 2
        gate, up = (x @ decoded(m.w_in[a:], m.s_in[b:], self.inner, self.dim).t().contiguous()
                    for a, b in ((0, 0), (self.inner, blocks)))
        h = gate / (1 + torch.exp(-gate)) * up
        return h @ decoded(m.w_out, m.s_out, self.dim, self.inner).t().contiguous(), r


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    import torch

    block = F8Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    mlp, r = (torch.randn((a.tokens, block.dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    positions = torch.arange(a.tokens, device="cuda") + 100000
    got, want = block.step(mlp, r, positions), block.step_fp64(mlp, r, positions)
    err = [float((x.double() - y).norm() / y.norm()) for x, y in zip(got, want)]
    print("against fp64: mlp %.4f, residual %.4f (relative)" % tuple(err))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        mlp, r = block.step(mlp, r, positions)
    end.record()
    torch.cuda.synchronize()
    print("%d token(s): %.1f us a step" % (a.tokens, 1e3 * start.elapsed_time(end) / a.steps))
    return err


if __name__ == "__main__":
    main()
