"""A decoder block of mixed precision, step by step through the library:

    python -m gemv_bit_unpack_amd.examples.mixed_block [--tokens 1] [--steps 8]

The attention part is stood in for by its two projections (an 8-bit input projection, a codebook-quantized output
projection of 3 bits per weight); the MLP is 8 experts in 8 bits, 2 for a token.  Between the parts run the norms with
the residual add, which hand 8-bit tokens to the 8-bit layers and 16-bit ones to the codebook layer:

    r, q, s = block_norm(mlp, r, post, pre, q8=True)     norm after the last MLP, residual add, norm before
    a       = Q8Linear.forward_q8(q, s)                  8-bit projection
    o       = VQLinear(a)                                codebook-quantized projection
    r, x    = block_norm(o, r, post, pre)                the same between the halves of the block
    mlp     = Q8Experts(x, ids, p)                       router's choice -> experts

Weights are random.  Prints the time of a step and how far it is from the same block in fp32 on the decoded weights.
"""
from __future__ import annotations

import argparse

import numpy as np


class MixedBlock:
    def __init__(self, dim=1024, inner=1792, experts=8, top=2, device="cuda", seed=0):
        import torch

        import gemv_bit_unpack_amd as vq

        self.vq, self.torch, self.top, self.experts = vq, torch, top, experts
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)
        self.norms = [0.1 * rnd(dim) + 1 for _ in range(4)]
        self.proj = vq.Q8Linear.from_weight(rnd(dim, dim) / dim ** 0.5)
        hr = np.random.default_rng(seed)
        desc = vq.make_desc(dim, dim, 8, 16, 8)
        self.out = vq.VQLinear.from_indices(
            desc, hr.integers(0, 1 << 16, (dim, dim // 8), dtype=np.uint32), hr.integers(0, 256, (dim, dim // 8), dtype=np.uint32),
            (rnd(1 << 16, 8) / dim ** 0.5).half(), (0.2 * rnd(256, 8) / dim ** 0.5).half(),
            (torch.rand((dim,), generator=g, device=device) + 0.5).half(), device=device)
        self.router = rnd(experts, dim) / dim ** 0.5
        wi, si = vq.q8_quantize(rnd(experts * 2 * inner, dim) / dim ** 0.5)
        wo, so = vq.q8_quantize(rnd(experts * dim, inner) / inner ** 0.5)
        self.mlp = vq.Q8Experts(wi[:, :dim].reshape(experts, 2 * inner, dim), si.reshape(experts, 2 * inner),
                                wo[:, :inner].reshape(experts, dim, inner), so.reshape(experts, dim))

    def route(self, x):
        torch = self.torch
        score, ids = (x.float() @ self.router.t()).topk(self.top, dim=1)
        return ids.to(torch.int32), torch.softmax(score, dim=1)

    def step(self, mlp, r):
        """(mlp output, residual) of the block before -> the same of this one; both [tokens, dim] bf16."""
        vq, n = self.vq, self.norms
        r, q, s = vq.block_norm(mlp, r, post="rms", post_weight=n[0], pre="rms", pre_weight=n[1], q8=True)
        o = self.out(self.proj.forward_q8(q, s))
        r, x = vq.block_norm(o, r, post="rms", post_weight=n[2], pre="rms", pre_weight=n[3])
        ids, p = self.route(x)
        return self.mlp(x, ids, p), r

    def step_fp32(self, mlp, r):
        """The same block in fp32 on the decoded weights, nothing rounded in between."""
        torch, vq, n = self.torch, self.vq, self.norms
        rms = lambda a, w: a / torch.sqrt((a * a).mean(1, keepdim=True) + 1e-6) * w
        dense = lambda w, s: w.float() * s.unsqueeze(-1)
        r = r.float() + rms(mlp.float(), n[0])
        a = rms(r, n[1]) @ dense(self.proj.w[:, :r.shape[1]], self.proj.scale).t()
        d = self.out
        o = a @ vq.dequant(d.desc, d.packed, d.cb1, d.cb2, d.scale).t()
        r = r + rms(o, n[2])
        x = rms(r, n[3])
        ids, p = self.route(x)
        y = torch.zeros_like(x)
        m = self.mlp
        for e in range(self.experts):
            tok, slot = (ids == e).nonzero(as_tuple=True)
            g, u = (x[tok] @ dense(m.w_in[e, :, :m.features], m.s_in[e]).t()).chunk(2, dim=1)
            h = g * torch.sigmoid(g) * u
            y[tok] += (h @ dense(m.w_out[e, :, :m.inner], m.s_out[e]).t()) * p[tok, slot].unsqueeze(1)
        return y, r


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    import torch

    block = MixedBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    mlp, r = (torch.randn((a.tokens, 1024), generator=g, device="cuda").bfloat16() for _ in range(2))
    got, want = block.step(mlp, r), block.step_fp32(mlp, r)
    err = [float((x.float() - y).norm() / y.norm()) for x, y in zip(got, want)]
    print("against fp32: mlp %.4f, residual %.4f (relative)" % tuple(err))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        mlp, r = block.step(mlp, r)
    end.record()
    torch.cuda.synchronize()
    print("%d token(s): %.1f us a step" % (a.tokens, 1e3 * start.elapsed_time(end) / a.steps))
    return err


if __name__ == "__main__":
    main()
