"""Rotary positions of queries and keys, with norms of their heads in the same pass (libvq's vq_rotate_heads).

    rope_frequencies(dim, base=10000.0, scaling=None) -> (frequencies, scale)
    Rotary(dim, base=10000.0, start=0, interleaved=False, scaling=None, device="cuda")
    rotate_heads(q, k, positions, rotary, norm="none", ...) -> (q', k')
Re-exported by the package's ``__init__``.
"""
from __future__ import annotations

import ctypes
import functools
import math


class HeadsDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("rot", ctypes.c_int32), ("start", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int), ("positions_64", ctypes.c_int32),
                ("position_stride", ctypes.c_int64), ("q_strides", ctypes.c_int64 * 3), ("k_strides", ctypes.c_int64 * 3),
                ("q_out_strides", ctypes.c_int64 * 3), ("k_out_strides", ctypes.c_int64 * 3), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float)]


def bind(lib):
    """Argument types of this entry point on a loaded libvq handle."""
    lib.vq_rotate_heads.argtypes = [ctypes.POINTER(HeadsDesc)] + [ctypes.c_void_p] * 11
    lib.vq_rotate_heads.restype = ctypes.c_int


from . import VQ_F32, _launch, _torch, lib  # noqa: E402
from .q8 import _KINDS, _code, _device, _ptr, _stream  # noqa: E402


def rope_frequencies(dim, base=10000.0, scaling=None):
    """Radians per position of the dim / 2 pairs of a rotated part, base^(-2 j / dim) as Python floats, and the factor on
    the rotated values (1.0 but for "yarn").

    ``scaling`` stretches a context for which the model was trained, by ``factor`` s >= 1:
        {"kind": "linear", "factor": s}   every pair at 1 / s of its speed (positions interpolated)
        {"kind": "ntk", "factor": s}      base * s^(dim / (dim - 2)): the slowest pair at 1 / s, the fastest as it was
        {"kind": "yarn", "factor": s, "length": L [, "fast": 32.0, "slow": 1.0, "scale": 0.1 ln s + 1]}
            pairs that turn more than ``fast`` times within L positions keep their speed, those that turn less than
            ``slow`` times get 1 / s of it, and a ramp over the pairs' numbers lies in between
        {"kind": "bands", "factor": s, "length": L, "low": a, "high": b}
            the same with a and b turns, and a ramp over the number of turns within L in between
        {"kind": "list", "factors": [..]} pair j at 1 / factors[j] of its speed [, "scale": ..]
    """
    dim, base = int(dim), float(base)
    if dim < 0 or dim % 2:
        raise ValueError("the rotated part must have an even number of values, got %d" % dim)
    if not (base > 0 and math.isfinite(base)):
        raise ValueError("base must be positive, got %r" % base)
    freqs = lambda b: [b ** (-2.0 * j / dim) for j in range(dim // 2)]
    if scaling is None:
        return freqs(base), 1.0
    opts = dict(scaling)
    kind = opts.pop("kind", None)
    allowed = {"linear": ("factor",), "ntk": ("factor",), "yarn": ("factor", "length", "fast", "slow", "scale"),
               "bands": ("factor", "length", "low", "high"), "list": ("factors", "scale")}
    if kind not in allowed:
        raise ValueError("scaling kind must be one of %s, got %r" % (tuple(allowed), kind))
    optional = ("fast", "slow", "scale")
    bad = [o for o in opts if o not in allowed[kind]] + [o for o in allowed[kind] if o not in opts and o not in optional]
    if bad:
        raise ValueError("%s scaling takes %s; missing or unknown: %s" % (kind, allowed[kind], bad))
    number = lambda what, low: _number(opts[what], what, low)
    scale = number("scale", 0.0) if "scale" in opts else 1.0
    if kind == "list":
        if len(opts["factors"]) != dim // 2:
            raise ValueError("factors must be %d, got %d" % (dim // 2, len(opts["factors"])))
        return [f / _number(x, "a factor", 0.0) for f, x in zip(freqs(base), opts["factors"])], scale
    s = number("factor", 0.0)
    if kind == "linear":
        return [f / s for f in freqs(base)], scale
    if kind == "ntk":
        return freqs(base * s ** (dim / (dim - 2.0)) if dim > 2 else base), scale
    length = number("length", 0.0)
    if kind == "bands":
        low, high = number("low", 0.0), number("high", 0.0)
        if not high > low:
            raise ValueError("high must be above low, got %r and %r" % (high, low))
        keep = [min(max((length * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in freqs(base)]
        return [k * f + (1 - k) * f / s for k, f in zip(keep, freqs(base))], scale
    fast, slow = (number(x, 0.0) if x in opts else d for x, d in (("fast", 32.0), ("slow", 1.0)))
    if base == 1.0:
        raise ValueError("yarn scaling needs a base other than 1")
    at = lambda turns: dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim - 1)
    ramp = [min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0) for j in range(dim // 2)]
    if "scale" not in opts:
        scale = 0.1 * math.log(s) + 1.0 if s > 1 else 1.0
    return [f / s * r + f * (1 - r) for f, r in zip(freqs(base), ramp)], scale


def _number(v, what, low):
    v = float(v)
    if not (v > low and math.isfinite(v)):
        raise ValueError("%s must be above %g and finite, got %r" % (what, low, v))
    return v


class Rotary:
    """The rotated part of a head, values ``start`` .. start + dim - 1, and its pairs' frequencies on the device:
    ``interleaved`` pairs are (2 j, 2 j + 1), others (j, j + dim / 2).  base and scaling as for rope_frequencies."""

    def __init__(self, dim, base=10000.0, start=0, interleaved=False, scaling=None, device="cuda"):
        torch = _torch()
        freqs, self.scale = rope_frequencies(dim, base, scaling)
        if start < 0:
            raise ValueError("start must not be negative, got %d" % start)
        self.dim, self.start, self.interleaved = int(dim), int(start), bool(interleaved)
        # turns per position; held here and not to be replaced: the calls take the pointer below
        self.freqs = torch.tensor([f / (2 * math.pi) for f in freqs], dtype=torch.float64, device=device)
        self._p, self._dev = self.freqs.data_ptr(), self.freqs.get_device()


def _view(shape, strides, what):
    """(batch, tokens, heads, dim) and the strides of the first three of [tokens, heads, dim] or [batch, tokens, heads, dim]
    whose heads are contiguous; strides None: of a contiguous tensor."""
    if len(shape) not in (3, 4):
        raise ValueError("%s must be [tokens, heads, dim] or [batch, tokens, heads, dim], got %s" % (what, tuple(shape)))
    *batch, n, h, d = shape
    if strides is None:
        strides = (n * h * d, h * d, d, 1)[4 - len(shape):]
    if strides[-1] != 1 and d > 1:
        raise ValueError("%s must have contiguous heads" % what)
    return (batch[0] if batch else 1, n, h, d), tuple(strides[:3]) if batch else (0,) + tuple(strides[:2])


@functools.lru_cache(maxsize=1024)
def _plan(q, k, positions, q_out, k_out, wide, rot, start, inter, kind, x_dtype, y_dtype, w_dtype, scale, eps, w_offset):
    """A vq_heads_desc, by reference (it is only read), of tensors given by their shapes and strides, checked once for all
    tensors alike.  Nothing here stands for a tensor itself or for its values."""
    (b, t, hq, d), qs = _view(*q, "q")
    hk, ks, kys = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        (kb, kt, hk, kd), ks = _view(*k, "k")
        if kt != t or kd != d or kb != b or len(k[0]) != len(q[0]):
            raise ValueError("k must have q's batch, tokens and dim, got %s and %s" % (tuple(k[0]), tuple(q[0])))
        kys = _view(k[0], k_out, "k_out")[1]
    qys = _view(q[0], q_out, "q_out")[1]
    if start + rot > d:
        raise ValueError("the rotated part ends at %d, a head at %d" % (start + rot, d))
    pos_stride = 0
    if positions is not None:
        shape, strides = positions
        if tuple(shape) != (t,) and (len(q[0]) != 4 or tuple(shape) != (b, t)):
            raise ValueError("positions must be [%d]%s, got %s" % (t, " or [%d, %d]" % (b, t) if len(q[0]) == 4 else "",
                                                                  tuple(shape)))
        if t > 1 and strides[-1] != 1:
            raise ValueError("positions of neighbouring tokens must be neighbours")
        if len(shape) == 2 and b > 1:
            pos_stride = strides[0]
    triple = ctypes.c_int64 * 3
    return ctypes.byref(HeadsDesc(b, t, hq, hk, d, rot, start, inter, kind, _code(x_dtype), _code(y_dtype),
                                  VQ_F32 if w_dtype is None else _code(w_dtype), wide, pos_stride, triple(*qs), triple(*ks),
                                  triple(*qys), triple(*kys), scale, eps, w_offset))


def _output(x, out, dtype, dev, what):
    """The output of x: (tensor, its strides or None for contiguous), a new one or `out`."""
    if out is None:
        return x.new_empty(x.shape, dtype=dtype), None
    if out.shape != x.shape:
        raise ValueError("%s must be %s, got %s" % (what, list(x.shape), tuple(out.shape)))
    if out.get_device() != dev or out.dtype is not dtype:
        raise ValueError("%s must be %s on device %d, is %s on %s" % (what, dtype, dev, out.dtype, out.device))
    return out, out.stride()


def rotate_heads(q, k, positions, rotary, *, norm="none", q_weight=None, q_bias=None, k_weight=None, k_bias=None, eps=1e-6,
                 weight_offset=0.0, out_dtype=None, q_out=None, k_out=None):
    """Norms of the heads of q and k and their rotary positions in one pass (vq_rotate_heads): (q', k').

    q [tokens, q heads, dim] or [batch, tokens, q heads, dim], k the same with its own number of heads, or None; any strides
    but of dim (views of one projection's output; [batch, heads, tokens, dim] transposed).  positions int32 or int64
    [tokens] or [batch, tokens] (one row for all batches with [tokens]; rows of any stride, expanded ones too); ``rotary``: a
    Rotary, or None for norms alone (positions are then not read).  norm: "none", "rms" or "layer" over each head, weights
    and biases [dim].  ``q_out``, ``k_out``: tensors to write into, of any strides, q and k themselves too; by default new
    contiguous ones of ``out_dtype`` (q's)."""
    torch = _torch()
    kind = _KINDS.get(norm)
    if kind is None:
        raise ValueError("norm must be one of %s" % (tuple(_KINDS),))
    dev, x_dtype = _device(q, "q"), q.dtype
    y_dtype = out_dtype or (x_dtype if q_out is None else q_out.dtype)
    q_out, q_strides = _output(q, q_out, y_dtype, dev, "q_out")
    k_view = k_strides = kp = kyp = None
    if k is not None:
        if k.dtype is not x_dtype or k.get_device() != dev:
            raise ValueError("k must have q's dtype and device, got %s on %s" % (k.dtype, k.device))
        k_out, k_strides = _output(k, k_out, y_dtype, dev, "k_out")
        k_view, kp, kyp = (k.shape, k.stride()), k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None or k_bias is not None:
        raise ValueError("k_out, k_weight and k_bias go with k")
    w_dtype, vecs = None, (None, None, None, None)
    if q_weight is not None or q_bias is not None or k_weight is not None or k_bias is not None:
        vecs, dim = [q_weight, q_bias, k_weight, k_bias], (q.shape[-1],)
        for i, v in enumerate(vecs):
            if v is not None:
                if w_dtype is None:
                    w_dtype = v.dtype
                elif v.dtype is not w_dtype:
                    raise TypeError("norm weights and biases must share one dtype")
                vecs[i] = _ptr(v, "a norm weight or bias", dim, dev)
    pos = pos_p = freqs_p = None
    wide = rot = start = inter = 0
    scale = 1.0
    if rotary is not None:
        rot, start, inter, scale, freqs_p = rotary.dim, rotary.start, int(rotary.interleaved), rotary.scale, rotary._p
        if rotary._dev != dev:
            raise ValueError("rotary must be on device %d, is on %s" % (dev, rotary.freqs.device))
        if positions is None:
            raise TypeError("positions must be given with a rotary")
        if positions.dtype is torch.int64:
            wide = 1
        elif positions.dtype is not torch.int32:
            raise TypeError("positions has dtype %s, expected int32 or int64" % positions.dtype)
        if positions.get_device() != dev:
            raise ValueError("positions must be on device %d, is on %s" % (dev, positions.device))
        pos, pos_p = (positions.shape, positions.stride()), positions.data_ptr()
    desc = _plan((q.shape, q.stride()), k_view, pos, q_strides, k_strides, wide, rot, start, inter, kind, x_dtype, y_dtype,
                 w_dtype, float(scale) + 0.0, float(eps) + 0.0, float(weight_offset) + 0.0)  # + 0.0: -0.0 is found as 0.0
    _launch(lib().vq_rotate_heads, dev, desc, q.data_ptr(), kp, pos_p, freqs_p, *vecs, q_out.data_ptr(), kyp, _stream(dev))
    return q_out, k_out
