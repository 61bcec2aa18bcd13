"""Layers in 8-bit floating point with block scales (libvq's vq_f8_*).

Argument marshalling only, as in the package's ``__init__`` (which re-exports every name here):
    f8_pad(w) -> float8_e4m3fn [N, q8_row_bytes(K)] (zero pads; w itself where K is whole already)
    f8_quantize(x, block_rows=1) -> (q, s)
    f8_gemm_workspace_bytes(m, n, k, gated), f8_linear_workspace_bytes(...), f8_mlp_workspace_bytes(m, d, i) -> int
    f8_gemm(q, s, w, sw, bias, k, gated=False, ws=None, y_dtype=..., out=None)
    f8_linear(x, w, sw, bias, ws, gated=False, y_dtype=None, out=None)
    f8_mlp(x, w_in, s_in, w_out, s_out, inner, ws, y_dtype=None, out=None)
plus the layer objects ``F8Linear`` and ``F8MLP``, whose calls take a workspace of their own each.

Values are torch.float8_e4m3fn; a token's scale stands for 128 columns, a weight's for a block of 128 x 128.  Token scales
are [ceil(K / 128), M], weight scales [ceil(N / 128), ceil(K / 128)]; weights of a gated product are the gate's rows and
the up projection's, each half with blocks of its own.
"""
from __future__ import annotations

import ctypes

BLOCK = 128


def bind(lib):
    """Argument types of these entry points on a loaded libvq handle."""
    vp, i32, i64, sz, e = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    szp = ctypes.POINTER(sz)
    args = {
        "vq_f8_quantize": [i32, i32, i32, vp, e, i64, vp, vp, vp],
        "vq_f8_gemm_workspace_bytes": [i32, i32, i32, i32, szp],
        "vq_f8_gemm": [i32, i32, i32, vp, vp, vp, vp, vp, i32, vp, e, vp, sz, vp],
        "vq_f8_linear_workspace_bytes": [i32, i32, i32, i32, szp],
        "vq_f8_linear": [i32, i32, i32, vp, e, i64, vp, vp, vp, i32, vp, e, vp, sz, vp],
        "vq_f8_mlp_workspace_bytes": [i32, i32, i32, szp],
        "vq_f8_mlp": [i32, i32, i32, vp, e, i64, vp, vp, vp, vp, vp, e, vp, sz, vp],
    }
    for name, types in args.items():
        f = getattr(lib, name)
        f.argtypes = types
        f.restype = ctypes.c_int


from . import _launch, _torch, lib  # noqa: E402
from .q8 import (_bytes_of, _code, _device, _out, _ptr, _rows, _stream, _tokens, _Weights, _workspace, _ws,  # noqa: E402
                 q8_row_bytes)


def f8_blocks(n: int) -> int:
    """Blocks of 128 that n rows or columns have."""
    return -(-n // BLOCK)


def _scales(n, k, gated=False):
    """Shape of the scales of weights with n outputs and k columns."""
    return ((2 if gated else 1) * f8_blocks(n), f8_blocks(k))


def f8_pad(w):
    """e4m3 values [..., k] laid out in rows of q8_row_bytes(k), zeros behind (done once, for weights)."""
    torch = _torch()
    if w.dtype != torch.float8_e4m3fn:
        raise TypeError("w has dtype %s, expected float8_e4m3fn" % w.dtype)
    pad = q8_row_bytes(w.shape[-1]) - w.shape[-1]
    if not pad:
        return w.contiguous()
    return torch.nn.functional.pad(w.view(torch.uint8), (0, pad)).view(torch.float8_e4m3fn)


def f8_quantize(x, block_rows=1, out=None):
    """Rows of x [M, K] (fp16, bf16 or fp32; any row stride) in e4m3: q [M, q8_row_bytes(K)] and s fp32, for tokens
    (block_rows 1) [ceil(K / 128), M], for weights (block_rows 128) [ceil(M / 128), ceil(K / 128)].  ``out``: the pair to
    write into."""
    torch = _torch()
    p, ld, code, dev = _rows(x, "x")
    m, k = x.shape
    row = q8_row_bytes(k)
    shape = (f8_blocks(m), f8_blocks(k)) if block_rows == BLOCK else (f8_blocks(k), m)
    q, s = out or (None, None)
    q, s = _out(q, (m, row), torch.float8_e4m3fn, x), _out(s, shape, torch.float32, x)
    _launch(lib().vq_f8_quantize, dev, m, k, int(block_rows), p, code, ld, _ptr(q, "q", (m, row), dev, torch.float8_e4m3fn),
            _ptr(s, "s", shape, dev, torch.float32), _stream(dev))
    return q, s


def f8_gemm_workspace_bytes(m: int, n: int, k: int, gated=False) -> int:
    return _bytes_of("vq_f8_gemm_workspace_bytes", m, n, k, int(bool(gated)))


def f8_linear_workspace_bytes(m: int, n: int, k: int, gated=False) -> int:
    return _bytes_of("vq_f8_linear_workspace_bytes", m, n, k, int(bool(gated)))


def f8_mlp_workspace_bytes(m: int, d: int, inner: int) -> int:
    return _bytes_of("vq_f8_mlp_workspace_bytes", m, d, inner)


def _outputs(w, gated):
    """Outputs of a product with weights w."""
    rows = w.shape[0]
    if gated and rows % 2:
        raise ValueError("a gated w must have an even number of rows, got %d" % rows)
    return rows // 2 if gated else rows


def _weights(w, sw, bias, n, k, gated, dev):
    torch = _torch()
    rows = 2 * n if gated else n
    return (_ptr(w, "w", (rows, q8_row_bytes(k)), dev, torch.float8_e4m3fn),
            _ptr(sw, "sw", _scales(n, k, gated), dev, torch.float32), _ptr(bias, "bias", (rows,), dev, torch.float16))


def f8_gemm(q, s, w, sw, bias, k, gated=False, ws=None, y_dtype=None, out=None):
    """y [M, N] = x w^T (+ bias) of tokens q, s and weights w, sw of k columns (as f8_quantize / f8_pad write them); gated:
    silu of the first N rows' product times that of the other N (vq_f8_gemm).

    ``ws``: a uint8 device buffer of f8_gemm_workspace_bytes(M, N, k, gated) (None: the product does not cut K).  Calls that
    share a workspace must be ordered (one stream)."""
    torch = _torch()
    dev = _device(q, "q")
    m, n, row = q.shape[0], _outputs(w, gated), q8_row_bytes(k)
    out = _out(out, (m, n), y_dtype or torch.bfloat16, q)
    _launch(lib().vq_f8_gemm, dev, m, n, k, _ptr(q, "q", (m, row), dev, torch.float8_e4m3fn),
            _ptr(s, "s", (f8_blocks(k), m), dev, torch.float32), *_weights(w, sw, bias, n, k, gated, dev), int(bool(gated)),
            _ptr(out, "out", (m, n), dev), _code(out.dtype), *_ws(ws, dev), _stream(dev))
    return out


def f8_linear(x, w, sw, bias, ws, gated=False, y_dtype=None, out=None):
    """f8_gemm on x [M, K] cut to 8 bits inside the call; ``ws``: a uint8 device buffer of f8_linear_workspace_bytes (None
    where that is 0); ``out`` does not overlap x."""
    p, ld, code, dev = _rows(x, "x")
    (m, k), n = x.shape, _outputs(w, gated)
    out = _out(out, (m, n), y_dtype or x.dtype, x)
    _launch(lib().vq_f8_linear, dev, m, n, k, p, code, ld, *_weights(w, sw, bias, n, k, gated, dev), int(bool(gated)),
            _ptr(out, "out", (m, n), dev), _code(out.dtype), *_ws(ws, dev), _stream(dev))
    return out


def f8_mlp(x, w_in, s_in, w_out, s_out, inner, ws, y_dtype=None, out=None):
    """A gated feed-forward layer (vq_f8_mlp): x [M, D], w_in [2 inner, ..] (gate rows first), w_out [D, ..]; ``ws``: a
    uint8 device buffer of f8_mlp_workspace_bytes."""
    p, ld, code, dev = _rows(x, "x")
    m, d = x.shape
    out = _out(out, (m, d), y_dtype or x.dtype, x)
    w_in, s_in, _ = _weights(w_in, s_in, None, inner, d, True, dev)
    w_out, s_out, _ = _weights(w_out, s_out, None, d, inner, False, dev)
    _launch(lib().vq_f8_mlp, dev, m, d, inner, p, code, ld, w_in, s_in, w_out, s_out, _ptr(out, "out", (m, d), dev),
            _code(out.dtype), *_ws(ws, dev), _stream(dev))
    return out


def _input(x, k, dev):
    """x [..., k] as rows: (rows, pointer, row stride, dtype code)."""
    rows = _tokens(x)
    p, ld, code, x_dev = _rows(rows, "x")
    if x_dev != dev or rows.shape[1] != k:
        raise ValueError("x must be [..., %d] on device %d, got %s on %s" % (k, dev, tuple(x.shape), x.device))
    return rows, p, ld, code


class F8Linear:
    """A linear layer in 8-bit floats: w float8_e4m3fn [N, K], fp32 scales [ceil(N / 128), ceil(K / 128)] of its blocks,
    optional fp16 bias.

    ``forward(x)`` cuts x [..., K] to 8 bits inside the call; ``forward_f8(q, s)`` takes tokens that f8_quantize cut."""

    def __init__(self, w, scale, bias=None):
        torch = _torch()
        n, k = self.out_features, self.in_features = w.shape
        self.w, self.scale, self.bias = f8_pad(w), scale, bias
        self._p = _Weights(w=(self.w, (n, q8_row_bytes(k)), torch.float8_e4m3fn),
                           scale=(scale, _scales(n, k), torch.float32), bias=(bias, (n,), torch.float16))

    @classmethod
    def from_weight(cls, w, bias=None):
        """From a dense weight [N, K] (fp16, bf16 or fp32 on the device), cut to 8 bits in blocks."""
        q, s = f8_quantize(w, BLOCK)
        return cls(q[:, :w.shape[1]], s, bias)

    def forward(self, x, y_dtype=None):
        n, k, w = self.out_features, self.in_features, self._p
        rows, p, ld, code = _input(x, k, w.dev)
        m = rows.shape[0]
        y = rows.new_empty((m, n), dtype=y_dtype or x.dtype)
        nbytes = f8_linear_workspace_bytes(m, n, k)
        ws, ws_p = _workspace(nbytes, rows)
        _launch(lib().vq_f8_linear, w.dev, m, n, k, p, code, ld, w.w, w.scale, w.bias, 0, y.data_ptr(), _code(y.dtype), ws_p,
                nbytes, _stream(w.dev))
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], n)

    __call__ = forward

    def forward_f8(self, q, s, y_dtype=None):
        torch = _torch()
        n, k, w = self.out_features, self.in_features, self._p
        m = q.shape[0]
        y = q.new_empty((m, n), dtype=y_dtype or torch.bfloat16)
        nbytes = f8_gemm_workspace_bytes(m, n, k)
        ws, ws_p = _workspace(nbytes, q)
        _launch(lib().vq_f8_gemm, w.dev, m, n, k, _ptr(q, "q", (m, q8_row_bytes(k)), w.dev, torch.float8_e4m3fn),
                _ptr(s, "s", (f8_blocks(k), m), w.dev, torch.float32), w.w, w.scale, w.bias, 0, y.data_ptr(),
                _code(y.dtype), ws_p, nbytes, _stream(w.dev))
        return y


class F8MLP:
    """A gated feed-forward layer in 8-bit floats: w_in float8_e4m3fn [2 I, D] (gate rows first), w_out [D, I], with the
    fp32 scales of their blocks s_in [2 ceil(I / 128), ceil(D / 128)] and s_out [ceil(D / 128), ceil(I / 128)]."""

    def __init__(self, w_in, s_in, w_out, s_out):
        torch = _torch()
        d, i = w_out.shape
        if tuple(w_in.shape) != (2 * i, d):  # the padded rows of another width could be as long
            raise ValueError("w_in must be %s, got %s" % ([2 * i, d], tuple(w_in.shape)))
        self.features, self.inner = d, i
        self.w_in, self.s_in, self.w_out, self.s_out = f8_pad(w_in), s_in, f8_pad(w_out), s_out
        e4m3 = torch.float8_e4m3fn
        self._p = _Weights(w_in=(self.w_in, (2 * i, q8_row_bytes(d)), e4m3), s_in=(s_in, _scales(i, d, True), torch.float32),
                           w_out=(self.w_out, (d, q8_row_bytes(i)), e4m3), s_out=(s_out, _scales(d, i), torch.float32))

    @classmethod
    def from_weights(cls, gate, up, out):
        """From dense weights gate and up [I, D] and out [D, I], cut to 8 bits in blocks."""
        torch = _torch()
        d, i = out.shape
        if tuple(gate.shape) != (i, d) or tuple(up.shape) != (i, d):  # behind the padding of rows it would not be seen
            raise ValueError("gate and up must be %s, got %s and %s" % ([i, d], tuple(gate.shape), tuple(up.shape)))
        (g, gs), (u, us), (o, os) = (f8_quantize(w, BLOCK) for w in (gate, up, out))
        w_in = torch.cat((g.view(torch.uint8), u.view(torch.uint8))).view(torch.float8_e4m3fn)
        return cls(w_in[:, :d], torch.cat((gs, us)), o[:, :i], os)

    def forward(self, x, y_dtype=None):
        """y [..., D] for x [..., D]."""
        d, i, w = self.features, self.inner, self._p
        rows, p, ld, code = _input(x, d, w.dev)
        m = rows.shape[0]
        y = rows.new_empty((m, d), dtype=y_dtype or x.dtype)
        nbytes = f8_mlp_workspace_bytes(m, d, i)
        ws, ws_p = _workspace(nbytes, rows)
        _launch(lib().vq_f8_mlp, w.dev, m, d, i, p, code, ld, w.w_in, w.s_in, w.w_out, w.s_out, y.data_ptr(), _code(y.dtype),
                ws_p, nbytes, _stream(w.dev))
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], d)

    __call__ = forward
