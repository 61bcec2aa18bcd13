"""8-bit operators of libvq: layers kept in 8 bits beside the codebook layers, their experts, and the norms in between.

Argument marshalling only, as in the package's ``__init__`` (which re-exports every name here):
    q8_row_bytes(k) -> int
    q8_pad(w) -> int8 [..., q8_row_bytes(k)] (zero pads; w itself where k is whole already)
    q8_quantize(x) -> (q, s)
    q8_gemm(q, s, w, sw, bias, k, ws=None, y_dtype=..., out=None)
    q8_linear(x, w, sw, bias, ws, y_dtype=None, out=None)
    expert_plan(ids, experts) -> (offsets, rows, pos)
    q8_gemm_grouped(offsets, rows, q, s, w, sw, bias, k, max_rows, gated=False, y_dtype=..., out=None)
    expert_combine(z, pos, p, y_dtype=..., out=None)
    q8_experts(x, ids, p, w_in, s_in, w_out, s_out, inner, ws, y_dtype=None, out=None)
    block_norm(z, residual=None, ...) -> (r, x) or (r, q, s)
plus the layer objects ``Q8Linear`` and ``Q8Experts``, which keep a workspace per device and stream as ``VQLinear`` does.
"""
from __future__ import annotations

import ctypes

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
_KINDS = {"none": NORM_NONE, "rms": NORM_RMS, "layer": NORM_LAYER}


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("dim", ctypes.c_int32), ("post", ctypes.c_int32), ("pre", ctypes.c_int32),
                ("z_dtype", ctypes.c_int), ("h_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("x_dtype", ctypes.c_int), ("gate_rows", ctypes.c_int32),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("gate_scale", ctypes.c_float), ("ldz", ctypes.c_int64), ("ldh", ctypes.c_int64)]


def bind(lib):
    """Argument types of the 8-bit entry points on a loaded libvq handle."""
    vp, i32, i64, sz, e = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    szp = ctypes.POINTER(sz)
    args = {
        "vq_q8_quantize": [i32, i32, vp, e, i64, vp, vp, vp],
        "vq_q8_gemm_workspace_bytes": [i32, i32, i32, szp],
        "vq_q8_gemm": [i32, i32, i32, vp, vp, vp, vp, vp, vp, e, vp, sz, vp],
        "vq_q8_linear_workspace_bytes": [i32, i32, i32, szp],
        "vq_q8_linear": [i32, i32, i32, vp, e, i64, vp, vp, vp, vp, e, vp, sz, vp],
        "vq_expert_plan": [i32, i32, i32, vp, vp, vp, vp, vp],
        "vq_q8_gemm_grouped": [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp, e, vp],
        "vq_expert_combine": [i32, i32, i32, i32, vp, vp, vp, vp, e, vp],
        "vq_q8_experts_workspace_bytes": [i32, i32, i32, i32, i32, szp],
        "vq_q8_experts": [i32, i32, i32, i32, i32, vp, e, i64, vp, vp, vp, vp, vp, vp, vp, e, vp, sz, vp],
        "vq_block_norm": [ctypes.POINTER(NormDesc)] + [vp] * 12,
    }
    for name, types in args.items():
        f = getattr(lib, name)
        f.argtypes = types
        f.restype = ctypes.c_int
    lib.vq_q8_row_bytes.argtypes = [i32]
    lib.vq_q8_row_bytes.restype = i64


from . import VQ_F32, _check, _dev_ptr, _dtype_code, _stream_ptr, _torch, lib  # noqa: E402


def _float_dtypes():
    torch = _torch()
    return (torch.float16, torch.bfloat16, torch.float32)


def _rows_ptr(t, what):
    """Pointer and row stride of a 2-d device tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-d, got %s" % (what, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % what)
    if t.dtype not in _float_dtypes():
        raise TypeError("%s has dtype %s, expected fp16, bf16 or fp32" % (what, t.dtype))
    m, k = t.shape
    if k > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % what)
    ld = t.stride(0) if m > 1 else k
    if ld < k:
        raise ValueError("%s must not have overlapping rows" % what)
    return ctypes.c_void_p(t.data_ptr()), ld


def _expect(t, what, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (what, list(shape), tuple(t.shape)))


def _same_device(ref, **others):
    for what, t in others.items():
        if t is not None and t.device != ref.device:
            raise ValueError("%s is on %s, expected %s" % (what, t.device, ref.device))


def _ws_args(ws):
    return (None, 0) if ws is None else (_dev_ptr(ws, "workspace"), ws.numel() * ws.element_size())


def _out(out, shape, dtype, device):
    if out is None:
        return _torch().empty(shape, dtype=dtype, device=device)
    _expect(out, "out", shape)
    return out


def q8_row_bytes(k: int) -> int:
    """Bytes of one row of an 8-bit matrix of k columns."""
    return int(lib().vq_q8_row_bytes(int(k)))


def q8_pad(w):
    """int8 values [..., k] laid out in rows of q8_row_bytes(k), zeros behind (done once, for weights)."""
    torch = _torch()
    if w.dtype != torch.int8:
        raise TypeError("w has dtype %s, expected int8" % w.dtype)
    pad = q8_row_bytes(w.shape[-1]) - w.shape[-1]
    return torch.nn.functional.pad(w, (0, pad)).contiguous() if pad else w.contiguous()


def q8_quantize(x, out=None):
    """Rows of x [M, K] (fp16, bf16 or fp32; any row stride) in 8 bits: (q int8 [M, q8_row_bytes(K)], s fp32 [M]).
    ``out``: the pair to write into."""
    torch = _torch()
    p, ld = _rows_ptr(x, "x")
    m, k = x.shape
    q, s = out or (None, None)
    q = _out(q, (m, q8_row_bytes(k)), torch.int8, x.device)
    s = _out(s, (m,), torch.float32, x.device)
    _same_device(x, q=q, s=s)
    _check(lib().vq_q8_quantize(m, k, p, _dtype_code(x.dtype), ld, _dev_ptr(q, "q", (torch.int8,)),
                                _dev_ptr(s, "s", (torch.float32,)), _stream_ptr(x.device)), "vq_q8_quantize")
    return q, s


def _bytes_of(fn, *shape):
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), fn)(*(int(v) for v in shape), ctypes.byref(n)), fn)
    return int(n.value)


def q8_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return _bytes_of("vq_q8_gemm_workspace_bytes", m, n, k)


def q8_linear_workspace_bytes(m: int, n: int, k: int) -> int:
    return _bytes_of("vq_q8_linear_workspace_bytes", m, n, k)


def q8_experts_workspace_bytes(tokens: int, top: int, experts: int, d: int, inner: int) -> int:
    return _bytes_of("vq_q8_experts_workspace_bytes", tokens, top, experts, d, inner)


def q8_gemm(q, s, w, sw, bias, k, ws=None, y_dtype=None, out=None):
    """y [M, N] = (q w^T) s sw (+ bias) of 8-bit rows of k columns (q and w as q8_quantize / q8_pad write them).

    ``ws``: a uint8 device buffer of q8_gemm_workspace_bytes(M, N, k) (None: the product does not cut K).  Calls that
    share a workspace must be ordered (one stream)."""
    torch = _torch()
    m, n = q.shape[0], w.shape[0]
    ld = q8_row_bytes(k)
    _expect(q, "q", (m, ld)), _expect(w, "w", (n, ld)), _expect(s, "s", (m,)), _expect(sw, "sw", (n,))
    _expect(bias, "bias", (n,))
    out = _out(out, (m, n), y_dtype or torch.bfloat16, q.device)
    _same_device(q, s=s, w=w, sw=sw, bias=bias, ws=ws, out=out)
    i8, f32 = (torch.int8,), (torch.float32,)
    _check(lib().vq_q8_gemm(m, n, k, _dev_ptr(q, "q", i8), _dev_ptr(s, "s", f32), _dev_ptr(w, "w", i8),
                            _dev_ptr(sw, "sw", f32), _dev_ptr(bias, "bias", (torch.float16,)), _dev_ptr(out, "out"),
                            _dtype_code(out.dtype), *_ws_args(ws), _stream_ptr(q.device)), "vq_q8_gemm")
    return out


def q8_linear(x, w, sw, bias, ws, y_dtype=None, out=None):
    """q8_gemm on x [M, K] cut to 8 bits inside the call; ``ws``: a uint8 device buffer of q8_linear_workspace_bytes."""
    torch = _torch()
    p, ld = _rows_ptr(x, "x")
    (m, k), n = x.shape, w.shape[0]
    _expect(w, "w", (n, q8_row_bytes(k))), _expect(sw, "sw", (n,)), _expect(bias, "bias", (n,))
    out = _out(out, (m, n), y_dtype or x.dtype, x.device)
    _same_device(x, w=w, sw=sw, bias=bias, ws=ws, out=out)
    _check(lib().vq_q8_linear(m, n, k, p, _dtype_code(x.dtype), ld, _dev_ptr(w, "w", (torch.int8,)),
                              _dev_ptr(sw, "sw", (torch.float32,)), _dev_ptr(bias, "bias", (torch.float16,)),
                              _dev_ptr(out, "out"), _dtype_code(out.dtype), *_ws_args(ws), _stream_ptr(x.device)),
           "vq_q8_linear")
    return out


def expert_plan(ids, experts: int):
    """Routing plan of int32 ids [T, top]: (offsets [experts + 1], rows [T * top], pos [T, top]); see vq_expert_plan."""
    torch = _torch()
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top], got %s" % (tuple(ids.shape),))
    t, top = ids.shape
    new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=ids.device)
    offsets, rows, pos = new(int(experts) + 1), new(t * top), new(t, top)
    _check(lib().vq_expert_plan(t, top, int(experts), _dev_ptr(ids, "ids", (torch.int32,)), _dev_ptr(offsets, "offsets"),
                                _dev_ptr(rows, "rows"), _dev_ptr(pos, "pos"), _stream_ptr(ids.device)), "vq_expert_plan")
    return offsets, rows, pos


def q8_gemm_grouped(offsets, rows, q, s, w, sw, bias, k, max_rows, gated=False, y_dtype=None, out=None):
    """The 8-bit product grouped by expert (vq_q8_gemm_grouped): y [max_rows, N] over sorted rows, w [E, N or 2 N, ..];
    ``rows`` None: sorted row r is row r of q.  Rows from offsets[E] on are not written."""
    torch = _torch()
    e, nw = w.shape[0], w.shape[1]
    if gated and nw % 2:
        raise ValueError("a gated w must have an even number of rows, got %d" % nw)
    n, ld = nw // 2 if gated else nw, q8_row_bytes(k)
    t = q.shape[0]
    _expect(q, "q", (t, ld)), _expect(s, "s", (t,)), _expect(w, "w", (e, nw, ld)), _expect(sw, "sw", (e, nw))
    _expect(bias, "bias", (e, nw)), _expect(offsets, "offsets", (e + 1,))
    if rows is not None and rows.numel() < max_rows:
        raise ValueError("rows must have at least max_rows = %d entries, got %d" % (max_rows, rows.numel()))
    out = _out(out, (max_rows, n), y_dtype or torch.float32, q.device)
    _same_device(q, offsets=offsets, rows=rows, s=s, w=w, sw=sw, bias=bias, out=out)
    i8, i32, f32 = (torch.int8,), (torch.int32,), (torch.float32,)
    _check(lib().vq_q8_gemm_grouped(e, max_rows, t, n, k, _dev_ptr(offsets, "offsets", i32), _dev_ptr(rows, "rows", i32),
                                    _dev_ptr(q, "q", i8), _dev_ptr(s, "s", f32), _dev_ptr(w, "w", i8),
                                    _dev_ptr(sw, "sw", f32), _dev_ptr(bias, "bias", (torch.float16,)),
                                    int(bool(gated)), _dev_ptr(out, "out"), _dtype_code(out.dtype),
                                    _stream_ptr(q.device)), "vq_q8_gemm_grouped")
    return out


def expert_combine(z, pos, p, y_dtype=None, out=None):
    """y [T, N] = sum_j p[t, j] z[pos[t, j]] of z fp32 [R, N], pos int32 and p fp32 [T, top]."""
    torch = _torch()
    t, top = pos.shape
    r, n = z.shape
    _expect(p, "p", (t, top))
    out = _out(out, (t, n), y_dtype or torch.float32, pos.device)
    _same_device(pos, z=z, p=p, out=out)
    _check(lib().vq_expert_combine(t, top, n, r, _dev_ptr(z, "z", (torch.float32,)), _dev_ptr(pos, "pos", (torch.int32,)),
                                   _dev_ptr(p, "p", (torch.float32,)), _dev_ptr(out, "out"), _dtype_code(out.dtype),
                                   _stream_ptr(pos.device)), "vq_expert_combine")
    return out


def q8_experts(x, ids, p, w_in, s_in, w_out, s_out, inner, ws, y_dtype=None, out=None):
    """A whole expert layer (vq_q8_experts): x [T, D], ids int32 and p fp32 [T, top], w_in [E, 2 inner, ..] (gate rows
    first), w_out [E, D, ..]; ``ws``: a uint8 device buffer of q8_experts_workspace_bytes."""
    torch = _torch()
    xp, ld = _rows_ptr(x, "x")
    t, d = x.shape
    e = w_in.shape[0]
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top], got %s" % (tuple(ids.shape),))
    top = ids.shape[1]
    _expect(ids, "ids", (t, top)), _expect(p, "p", (t, top))
    _expect(w_in, "w_in", (e, 2 * inner, q8_row_bytes(d))), _expect(s_in, "s_in", (e, 2 * inner))
    _expect(w_out, "w_out", (e, d, q8_row_bytes(inner))), _expect(s_out, "s_out", (e, d))
    out = _out(out, (t, d), y_dtype or x.dtype, x.device)
    _same_device(x, ids=ids, p=p, w_in=w_in, s_in=s_in, w_out=w_out, s_out=s_out, ws=ws, out=out)
    i8, f32 = (torch.int8,), (torch.float32,)
    _check(lib().vq_q8_experts(t, top, e, d, inner, xp, _dtype_code(x.dtype), ld, _dev_ptr(ids, "ids", (torch.int32,)),
                               _dev_ptr(p, "p", f32), _dev_ptr(w_in, "w_in", i8), _dev_ptr(s_in, "s_in", f32),
                               _dev_ptr(w_out, "w_out", i8), _dev_ptr(s_out, "s_out", f32), _dev_ptr(out, "out"),
                               _dtype_code(out.dtype), *_ws_args(ws), _stream_ptr(x.device)), "vq_q8_experts")
    return out


def block_norm(z, residual=None, *, post="none", post_weight=None, post_bias=None, pre="rms", pre_weight=None,
               pre_bias=None, gate=None, gate_rows=1, res_scale=1.0, gate_scale=1.0, eps=1e-6, weight_offset=0.0,
               x_dtype=None, q8=False, r_out=None, keep_r=True):
    """Between two blocks, in one pass (vq_block_norm):

        r = res_scale * residual + gate_scale * gate * N_post(z),    x = N_pre(r)

    z, residual [M, D] (any row strides); post / pre: "none", "rms" or "layer"; weights and biases [D]; gate [D], or
    [ceil(M / gate_rows), D] with one row for every gate_rows rows.  Returns (r, x), or with ``q8`` (r, q, s): x in
    8 bits.  r has the residual's dtype (z's without one); ``r_out`` may be the residual itself; ``keep_r=False``
    returns None for it.  x_dtype defaults to z's."""
    torch = _torch()
    if post not in _KINDS or pre not in _KINDS:
        raise ValueError("post and pre must be one of %s" % (tuple(_KINDS),))
    zp, ldz = _rows_ptr(z, "z")
    m, d = z.shape
    hp, ldh = (None, d) if residual is None else _rows_ptr(residual, "residual")
    _expect(residual, "residual", (m, d))
    vecs = [v for v in (post_weight, post_bias, pre_weight, pre_bias) if v is not None]
    for v in vecs:
        _expect(v, "a norm weight or bias", (d,))
        if v.dtype != vecs[0].dtype:
            raise TypeError("norm weights and biases must share one dtype")
    if gate is not None:
        if gate.dim() == 1:
            gate, gate_rows = gate.unsqueeze(0), max(m, 1)
        if gate_rows < 1:
            raise ValueError("gate_rows must be at least 1, got %d" % gate_rows)
        _expect(gate, "gate", (-(-m // gate_rows), d))
    r_dtype = z.dtype if residual is None else residual.dtype
    r = None
    if keep_r or r_out is not None:
        r = _out(r_out, (m, d), r_dtype, z.device)
    x = q = s = None
    if q8:
        q = torch.empty((m, q8_row_bytes(d)), dtype=torch.int8, device=z.device)
        s = torch.empty((m,), dtype=torch.float32, device=z.device)
    else:
        x = torch.empty((m, d), dtype=x_dtype or z.dtype, device=z.device)
    _same_device(z, residual=residual, post_weight=post_weight, post_bias=post_bias, pre_weight=pre_weight,
                 pre_bias=pre_bias, gate=gate, r_out=r_out)
    code = lambda t: VQ_F32 if t is None else _dtype_code(t.dtype)
    desc = NormDesc(m, d, _KINDS[post], _KINDS[pre], code(z), _dtype_code(r_dtype), code(vecs[0] if vecs else None),
                    code(gate), code(x), min(int(gate_rows), 2 ** 31 - 1), eps, weight_offset, res_scale, gate_scale,
                    ldz, ldh)
    _check(lib().vq_block_norm(ctypes.byref(desc), zp, hp, _dev_ptr(post_weight, "post_weight"),
                               _dev_ptr(post_bias, "post_bias"), _dev_ptr(pre_weight, "pre_weight"),
                               _dev_ptr(pre_bias, "pre_bias"), _dev_ptr(gate, "gate"), _dev_ptr(r, "r", (r_dtype,)),
                               _dev_ptr(x, "x"), _dev_ptr(q, "q"), _dev_ptr(s, "s"), _stream_ptr(z.device)),
           "vq_block_norm")
    return (r, q, s) if q8 else (r, x)


_stream_ws = {}


def _stream_workspace(nbytes, device):
    """A workspace kept per (device, current stream), grown on demand (None for 0 bytes)."""
    torch = _torch()
    if nbytes == 0:
        return None
    key = (device.index if device.index is not None else torch.cuda.current_device(),
           torch.cuda.current_stream(device).cuda_stream)
    ws = _stream_ws.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _stream_ws[key] = ws
    return ws


class Q8Linear:
    """A linear layer in 8 bits: w int8 [N, K], one fp32 scale per output channel, optional fp16 bias.

    ``forward(x)`` cuts x [..., K] to 8 bits per token inside the call; ``forward_q8(q, s)`` takes tokens that are in
    8 bits already (block_norm, q8_quantize)."""

    def __init__(self, w, scale, bias=None):
        self.out_features, self.in_features = w.shape
        self.w, self.scale, self.bias = q8_pad(w), scale, bias

    @classmethod
    def from_weight(cls, w, bias=None):
        """From a dense weight [N, K] (fp16, bf16 or fp32 on the device), cut to 8 bits per row."""
        q, s = q8_quantize(w)
        return cls(q[:, :w.shape[1]], s, bias)

    def forward(self, x, y_dtype=None):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1])
        if x2.shape[1] > 1 and x2.stride(1) != 1:
            x2 = x2.contiguous()
        ws = _stream_workspace(q8_linear_workspace_bytes(x2.shape[0], self.out_features, self.in_features), x2.device)
        return q8_linear(x2, self.w, self.scale, self.bias, ws, y_dtype).reshape(*lead, self.out_features)

    __call__ = forward

    def forward_q8(self, q, s, y_dtype=None):
        ws = _stream_workspace(q8_gemm_workspace_bytes(q.shape[0], self.out_features, self.in_features), q.device)
        return q8_gemm(q, s, self.w, self.scale, self.bias, self.in_features, ws, y_dtype)


class Q8Experts:
    """An expert layer in 8 bits: w_in int8 [E, 2 I, D] (gate rows first), w_out int8 [E, D, I], fp32 channel scales
    s_in [E, 2 I] and s_out [E, D]."""

    def __init__(self, w_in, s_in, w_out, s_out):
        self.experts, self.inner = w_in.shape[0], w_out.shape[2]
        self.w_in, self.s_in, self.w_out, self.s_out = q8_pad(w_in), s_in, q8_pad(w_out), s_out

    def forward(self, x, ids, p, y_dtype=None):
        """y [..., D] for x [..., D] and its tokens' expert ids (int32) and weights (fp32) [tokens, top]."""
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1])
        if x2.shape[1] > 1 and x2.stride(1) != 1:
            x2 = x2.contiguous()
        ws = _stream_workspace(q8_experts_workspace_bytes(x2.shape[0], ids.shape[1], self.experts, x2.shape[1],
                                                          self.inner), x2.device)
        y = q8_experts(x2, ids, p, self.w_in, self.s_in, self.w_out, self.s_out, self.inner, ws, y_dtype)
        return y.reshape(*lead, x2.shape[1])

    __call__ = forward
