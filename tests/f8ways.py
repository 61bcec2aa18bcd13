"""The ways in which the 8-bit float products are computed, which shapes take them, and operands whose sums are exact in all of
them."""
from __future__ import annotations

import ctypes

import torch

E4 = torch.float8_e4m3fn

WAYS = ("stream1", "stream2", "32x32", "32x64", "64x64", "64x128", "128x128", "128x128 pair", "256x256")


class _Plan(ctypes.Structure):
    _fields_ = [("way", ctypes.c_int32), ("splits", ctypes.c_int32), ("cut", ctypes.c_bool)]


def _name(p, gated, wide):
    return "%s%s%s %s %s" % (WAYS[p.way], ", K cut" if p.splits > 1 else "", ", tokens cut inside" if p.cut else "",
                             "gated" if gated else "dense", "fp16 operands" if wide else "e4m3 operands")


def plan(lib, m, n, k, gated, wide, may_cut):
    """The way of a product: wide, of fp32 outputs (or hidden rows); may_cut, of tokens that are not in 8 bits yet."""
    f = getattr(lib, "_ZN3vqi7f8_planEiiibbb")  # vqi::f8_plan
    f.restype, f.argtypes = _Plan, [ctypes.c_int32] * 3 + [ctypes.c_bool] * 3
    return _name(f(m, n, k, gated, wide, may_cut), gated, wide)


def ways(lib, m, n, k, gated):
    """Every way that the calls of this shape take."""
    return {plan(lib, m, n, k, gated, wide, cut) for wide in (False, True) for cut in (False, True)}


def writes_hidden(lib, m, d, i):
    """Whether the gated product of a feed-forward layer writes its hidden rows in 8 bits itself."""
    f = getattr(lib, "_ZN3vqi7f8_planEiiibbb")
    f.restype, f.argtypes = _Plan, [ctypes.c_int32] * 3 + [ctypes.c_bool] * 3
    p = f(m, i, d, True, True, True)
    big = getattr(lib, "_ZN3vqi11f8_big_planEiiiRNS_6F8PlanE")  # vqi::f8_big_plan
    big.restype, big.argtypes = ctypes.c_bool, [ctypes.c_int32] * 3 + [ctypes.POINTER(_Plan)]
    return big(m, i, d, ctypes.byref(p))


# (m, n, k, gated): between them every way that the rule takes, with odd sizes; and larger ones of the same ways
SHAPES = [(1, 157, 6228, False), (1, 681, 13475, False), (2, 153, 7190, False), (2, 551, 8150, False), (2, 4180, 712, False),
          (5, 151, 703, False), (17, 155, 4030, False), (17, 163, 4625, False), (18, 153, 737, False), (65, 16933, 919, False),
          (71, 16892, 22718, False), (128, 8192, 28672, False), (129, 23261, 704, False), (131, 22687, 1540, False),
          (326, 196, 6960, False), (683, 156, 23556, False), (1030, 9001, 1000, False), (1357, 170, 807, False),
          (2235, 669, 704, False), (2364, 198, 723, False), (2680, 844, 28292, False),
          (1, 700, 9000, True), (5, 151, 703, True), (18, 153, 737, True), (64, 14336, 4096, True), (66, 8628, 906, True),
          (67, 16698, 707, True), (143, 11288, 1628, True), (390, 312, 785, True), (611, 401, 700, True),
          (1100, 9001, 900, True), (2749, 267, 728, True)]

# (m, d, i) of feed-forward layers, and whether the hidden rows leave the gated product in 8 bits
LAYERS = [(1, 300, 700, False), (3, 400, 5001, False), (40, 512, 2000, False), (77, 256, 9300, True), (129, 300, 10001, True),
          (300, 264, 10001, True), (700, 650, 5500, True), (2049, 384, 6001, True)]


def tokens(g, m, k, dtype):
    """x [m, k] of `dtype` that its 8 bits hold: in each block of 128 columns 64 z 2^e, z whole and 7 at most, one of them 7, so
    that the block's scale is 2^e."""
    blocks = -(-k // 128)
    z = torch.randint(-7, 8, (m, blocks * 128), generator=g, device="cuda").float()
    at = torch.arange(blocks, device="cuda") * 128
    z[:, at] = torch.where(z[:, at] < 0, -7.0, 7.0)  # the first column of a block is always there
    e = torch.randint(-2, 3, (m, blocks), generator=g, device="cuda").float()
    return (z * 64 * torch.exp2(e).repeat_interleave(128, dim=1))[:, :k].to(dtype)


def weights(g, n, k, halves=1, shift=0):
    """(e4m3 [halves n, k], scales, values in fp64): whole numbers up to 4, scales 2^(shift - 2 .. shift + 2)."""
    nb, kb = -(-n // 128), -(-k // 128)
    w = torch.randint(-4, 5, (halves * n, k), generator=g, device="cuda", dtype=torch.int8)
    s = torch.exp2(torch.randint(shift - 2, shift + 3, (halves * nb, kb), generator=g, device="cuda").float())
    full = torch.cat([p.repeat_interleave(128, 0)[:n] for p in s.split(nb)]).double().repeat_interleave(128, 1)[:, :k]
    return w.float().to(E4), s, full.mul_(w)


def unit_shift(k):
    """The weights' shift for which sums over k columns have a spread near 2: tokens spread by 64 * 4.3 * 2^e (root mean
    square of 2^e: 2.1), weights by 2.6 * 2.1."""
    import math

    return 1 - round(math.log2(64 * 4.3 * 2.1 * 2.6 * 2.1 * k ** 0.5))
