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
plus the layer objects ``Q8Linear`` and ``Q8Experts``, whose calls take a workspace of their own each.
"""
from __future__ import annotations

import ctypes
import functools

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ONE_MAX_K = 48128  # VQ_Q8_ONE_MAX_K: up to this K one token's q8_linear takes no workspace
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


from . import VQ_BF16, VQ_F16, VQ_F32, _check, _launch, _torch, lib  # noqa: E402

_codes = {}


def _code(dt):
    """vq_dtype of a torch dtype."""
    if not _codes:
        torch = _torch()
        _codes.update({torch.float16: VQ_F16, torch.bfloat16: VQ_BF16, torch.float32: VQ_F32})
    code = _codes.get(dt)
    if code is None:
        raise TypeError("unsupported dtype %s, expected fp16, bf16 or fp32" % dt)
    return code


def _stream(dev):
    """Handle of the current stream of device index dev (torch.cuda.current_stream(dev).cuda_stream, without its object)."""
    return _torch()._C._cuda_getCurrentRawStream(dev)


@functools.lru_cache(maxsize=1024)
def _norm_desc(*fields):
    """A vq_norm_desc, by reference (it is only read); plain numbers only, which are what they compare as: a tensor would
    be found again by its identity, with the value that it had then."""
    return ctypes.byref(NormDesc(*fields))


def _device(t, what):
    """Device index of a device tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a device tensor" % what)
    return dev


def _rows(t, what):
    """(pointer, row stride, dtype code, device index) of a 2-d device tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-d, got %s" % (what, tuple(t.shape)))
    dev = _device(t, what)
    m, k = t.shape
    if t.is_contiguous():
        return t.data_ptr(), k, _code(t.dtype), dev
    ld, one = t.stride()
    if k > 1 and one != 1:
        raise ValueError("%s must have contiguous rows" % what)
    if m <= 1:
        ld = k
    if ld < k:
        raise ValueError("%s must not have overlapping rows" % what)
    return t.data_ptr(), ld, _code(t.dtype), dev


def _ptr(t, what, shape, dev, dtype=None):
    """Pointer of a contiguous tensor of the given shape (None: any) on device dev (None for no tensor)."""
    if t is None:
        return None
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError("%s must be %s, got %s" % (what, list(shape), tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on device %d, is on %s" % (what, dev, t.device))
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (what, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def _ws(ws, dev):
    """(pointer, bytes) of a workspace."""
    return (None, 0) if ws is None else (_ptr(ws, "workspace", None, dev), ws.numel() * ws.element_size())


def _like(t, dtype):
    """A new tensor of t's shape, contiguous."""
    if t.dtype is dtype and t.is_contiguous():
        return _torch().empty_like(t)
    return t.new_empty(t.shape, dtype=dtype)


def _out(out, shape, dtype, like):
    """An output of this shape: `out` itself, checked by _ptr later, or a new tensor on like's device."""
    return like.new_empty(shape, dtype=dtype) if out is None else out


@functools.lru_cache(maxsize=4096)
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
    p, ld, code, dev = _rows(x, "x")
    m, k = x.shape
    row = q8_row_bytes(k)
    q, s = out or (None, None)
    q, s = _out(q, (m, row), torch.int8, x), _out(s, (m,), torch.float32, x)
    _launch(lib().vq_q8_quantize, dev, m, k, p, code, ld, _ptr(q, "q", (m, row), dev, torch.int8),
            _ptr(s, "s", (m,), dev, torch.float32), _stream(dev))
    return q, s


@functools.lru_cache(maxsize=4096)
def _bytes_of(fn, *shape):
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), fn)(*shape, ctypes.byref(n)), fn)
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
    dev = _device(q, "q")
    m, n, row = q.shape[0], w.shape[0], q8_row_bytes(k)
    out = _out(out, (m, n), y_dtype or torch.bfloat16, q)
    f32 = torch.float32
    _launch(lib().vq_q8_gemm, dev, m, n, k, _ptr(q, "q", (m, row), dev, torch.int8), _ptr(s, "s", (m,), dev, f32),
            _ptr(w, "w", (n, row), dev, torch.int8), _ptr(sw, "sw", (n,), dev, f32),
            _ptr(bias, "bias", (n,), dev, torch.float16), _ptr(out, "out", (m, n), dev), _code(out.dtype),
            *_ws(ws, dev), _stream(dev))
    return out


def q8_linear(x, w, sw, bias, ws, y_dtype=None, out=None):
    """q8_gemm on x [M, K] cut to 8 bits inside the call; ``ws``: a uint8 device buffer of q8_linear_workspace_bytes
    (None is taken for M = 1 and K <= ONE_MAX_K)."""
    torch = _torch()
    p, ld, code, dev = _rows(x, "x")
    (m, k), n = x.shape, w.shape[0]
    out = _out(out, (m, n), y_dtype or x.dtype, x)
    _launch(lib().vq_q8_linear, dev, m, n, k, p, code, ld, _ptr(w, "w", (n, q8_row_bytes(k)), dev, torch.int8),
            _ptr(sw, "sw", (n,), dev, torch.float32), _ptr(bias, "bias", (n,), dev, torch.float16),
            _ptr(out, "out", (m, n), dev), _code(out.dtype), *_ws(ws, dev), _stream(dev))
    return out


def expert_plan(ids, experts: int):
    """Routing plan of int32 ids [T, top]: (offsets [experts + 1], rows [T * top], pos [T, top]); see vq_expert_plan."""
    torch = _torch()
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top], got %s" % (tuple(ids.shape),))
    dev = _device(ids, "ids")
    t, top = ids.shape
    # refused sizes are the library's to name; it is given no buffer for them
    offsets = ids.new_empty((max(int(experts), 0) + 1,), dtype=torch.int32)
    rows, pos = ids.new_empty((t * top,), dtype=torch.int32), ids.new_empty((t, top), dtype=torch.int32)
    _launch(lib().vq_expert_plan, dev, t, top, int(experts), _ptr(ids, "ids", (t, top), dev, torch.int32),
            offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(), _stream(dev))
    return offsets, rows, pos


def q8_gemm_grouped(offsets, rows, q, s, w, sw, bias, k, max_rows, gated=False, y_dtype=None, out=None):
    """The 8-bit product grouped by expert (vq_q8_gemm_grouped): y [max_rows, N] over sorted rows, w [E, N or 2 N, ..];
    ``rows`` None: sorted row r is row r of q.  Rows from offsets[E] on are not written."""
    torch = _torch()
    dev = _device(q, "q")
    e, nw = w.shape[0], w.shape[1]
    if gated and nw % 2:
        raise ValueError("a gated w must have an even number of rows, got %d" % nw)
    n, row, t = nw // 2 if gated else nw, q8_row_bytes(k), q.shape[0]
    if rows is not None and rows.numel() < max_rows:
        raise ValueError("rows must have at least max_rows = %d entries, got %d" % (max_rows, rows.numel()))
    out = _out(out, (max_rows, n), y_dtype or torch.float32, q)
    i8, i32, f32 = torch.int8, torch.int32, torch.float32
    _launch(lib().vq_q8_gemm_grouped, dev, e, max_rows, t, n, k, _ptr(offsets, "offsets", (e + 1,), dev, i32),
            _ptr(rows, "rows", None, dev, i32), _ptr(q, "q", (t, row), dev, i8), _ptr(s, "s", (t,), dev, f32),
            _ptr(w, "w", (e, nw, row), dev, i8), _ptr(sw, "sw", (e, nw), dev, f32),
            _ptr(bias, "bias", (e, nw), dev, torch.float16), int(bool(gated)), _ptr(out, "out", (max_rows, n), dev),
            _code(out.dtype), _stream(dev))
    return out


def expert_combine(z, pos, p, y_dtype=None, out=None):
    """y [T, N] = sum_j p[t, j] z[pos[t, j]] of z fp32 [R, N], pos int32 and p fp32 [T, top]."""
    torch = _torch()
    dev = _device(pos, "pos")
    (t, top), (r, n) = pos.shape, z.shape
    out = _out(out, (t, n), y_dtype or torch.float32, pos)
    _launch(lib().vq_expert_combine, dev, t, top, n, r, _ptr(z, "z", (r, n), dev, torch.float32),
            _ptr(pos, "pos", (t, top), dev, torch.int32), _ptr(p, "p", (t, top), dev, torch.float32),
            _ptr(out, "out", (t, n), dev), _code(out.dtype), _stream(dev))
    return out


def q8_experts(x, ids, p, w_in, s_in, w_out, s_out, inner, ws, y_dtype=None, out=None):
    """A whole expert layer (vq_q8_experts): x [T, D], ids int32 and p fp32 [T, top], w_in [E, 2 inner, ..] (gate rows
    first), w_out [E, D, ..]; ``ws``: a uint8 device buffer of q8_experts_workspace_bytes."""
    torch = _torch()
    xp, ld, code, dev = _rows(x, "x")
    t, d = x.shape
    e = w_in.shape[0]
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top], got %s" % (tuple(ids.shape),))
    top = ids.shape[1]
    out = _out(out, (t, d), y_dtype or x.dtype, x)
    i8, f32 = torch.int8, torch.float32
    _launch(lib().vq_q8_experts, dev, t, top, e, d, inner, xp, code, ld, _ptr(ids, "ids", (t, top), dev, torch.int32),
            _ptr(p, "p", (t, top), dev, f32), _ptr(w_in, "w_in", (e, 2 * inner, q8_row_bytes(d)), dev, i8),
            _ptr(s_in, "s_in", (e, 2 * inner), dev, f32), _ptr(w_out, "w_out", (e, d, q8_row_bytes(inner)), dev, i8),
            _ptr(s_out, "s_out", (e, d), dev, f32), _ptr(out, "out", (t, d), dev), _code(out.dtype), *_ws(ws, dev),
            _stream(dev))
    return out


def block_norm(z, residual=None, *, post="none", post_weight=None, post_bias=None, pre="rms", pre_weight=None,
               pre_bias=None, gate=None, gate_rows=1, res_scale=1.0, gate_scale=1.0, eps=1e-6, weight_offset=0.0,
               x_dtype=None, q8=False, r_out=None, keep_r=True):
    """Between two blocks, in one pass (vq_block_norm):

        r = res_scale * residual + gate_scale * gate * N_post(z),    x = N_pre(r)

    z, residual [M, D] (any row strides) or [..., D], M rows in all; post / pre: "none", "rms" or "layer"; weights and
    biases [D]; gate [D], or [ceil(M / gate_rows), D] with one row for every gate_rows rows.  Returns (r, x) of z's shape,
    or with ``q8`` (r, q, s): x in 8 bits, M rows.  r has the residual's dtype (z's without one); ``r_out`` may be the
    residual itself; ``keep_r=False`` returns None for it.  x_dtype defaults to z's."""
    if z.dim() > 2 or z.dim() == 1:
        for what, t in (("residual", residual), ("r_out", r_out)):
            if t is not None and t.shape != z.shape:
                raise ValueError("%s must be %s, got %s" % (what, list(z.shape), tuple(t.shape)))
        if r_out is not None and not r_out.is_contiguous():
            raise ValueError("r_out must be contiguous")
        flat = lambda t: None if t is None else _tokens(t)
        r, *x = block_norm(flat(z), flat(residual), post=post, post_weight=post_weight, post_bias=post_bias, pre=pre,
                           pre_weight=pre_weight, pre_bias=pre_bias, gate=gate, gate_rows=gate_rows, res_scale=res_scale,
                           gate_scale=gate_scale, eps=eps, weight_offset=weight_offset, x_dtype=x_dtype, q8=q8,
                           r_out=flat(r_out), keep_r=keep_r)
        r = r_out if r is None or r_out is not None else r.reshape(z.shape)
        return (r, *x) if q8 else (r, x[0].reshape(z.shape))
    kinds = _KINDS.get(post), _KINDS.get(pre)
    if None in kinds:
        raise ValueError("post and pre must be one of %s" % (tuple(_KINDS),))
    zp, ldz, z_code, dev = _rows(z, "z")
    m, d = z.shape
    hp, ldh, h_code, r_dtype = None, d, z_code, z.dtype
    if residual is not None:
        if residual.shape != z.shape:
            raise ValueError("residual must be %s, got %s" % ([m, d], tuple(residual.shape)))
        hp, ldh, h_code, h_dev = _rows(residual, "residual")
        if h_dev != dev:
            raise ValueError("residual must be on device %d, is on %s" % (dev, residual.device))
        r_dtype = residual.dtype
    w_dtype, vecs = None, [None] * 4
    for i, v in enumerate((post_weight, post_bias, pre_weight, pre_bias)):
        if v is not None:
            if w_dtype is None:
                w_dtype = v.dtype
            elif v.dtype is not w_dtype:
                raise TypeError("norm weights and biases must share one dtype")
            vecs[i] = _ptr(v, "a norm weight or bias", (d,), dev)
    gate_p, gate_code = None, VQ_F32
    if gate is not None:
        if gate.dim() == 1:
            gate_rows, shape = max(m, 1), (d,)
        elif gate_rows < 1:
            raise ValueError("gate_rows must be at least 1, got %d" % gate_rows)
        else:
            shape = (-(-m // gate_rows), d)
        gate_p, gate_code = _ptr(gate, "gate", shape, dev), _code(gate.dtype)
    r, r_p = r_out, None
    if r_out is not None:
        r_p = _ptr(r_out, "r_out", (m, d), dev, r_dtype)
    elif keep_r:
        r = _like(z if residual is None else residual, r_dtype)
        r_p = r.data_ptr()
    x = q = s = x_p = q_p = s_p = None
    x_code = VQ_F32
    if q8:
        torch = _torch()
        q, s = z.new_empty((m, q8_row_bytes(d)), dtype=torch.int8), z.new_empty((m,), dtype=torch.float32)
        q_p, s_p = q.data_ptr(), s.data_ptr()
    else:
        x = _like(z, x_dtype or z.dtype)
        x_p, x_code = x.data_ptr(), _code(x.dtype)
    desc = _norm_desc(m, d, *kinds, z_code, h_code, VQ_F32 if w_dtype is None else _code(w_dtype), gate_code, x_code,
                      min(int(gate_rows), 2 ** 31 - 1), float(eps) + 0.0, float(weight_offset) + 0.0,
                      float(res_scale) + 0.0, float(gate_scale) + 0.0, ldz, ldh)  # + 0.0: -0.0 is found as 0.0
    _launch(lib().vq_block_norm, dev, desc, zp, hp, *vecs, gate_p, r_p, x_p, q_p, s_p, _stream(dev))
    return (r, q, s) if q8 else (r, x)


def _workspace(nbytes, like):
    """(workspace on like's device, its pointer) for one call; (None, None) for 0 bytes.

    A call is several launches that share it, so it belongs to that call alone: the allocator hands its memory out again
    only behind these launches on their stream, gives calls of other threads other memory, and calls under capture memory
    that the graph keeps."""
    if nbytes == 0:
        return None, None
    ws = like.new_empty(nbytes, dtype=_torch().uint8)
    return ws, ws.data_ptr()


def _tokens(x):
    """x [..., K] as rows [M, K] (copied only where its rows are not contiguous, or overlap as those of an expanded view)."""
    if x.dim() != 2:
        x = x.reshape(-1, x.shape[-1])
    if x.is_contiguous():
        return x
    (m, k), (ld, one) = x.shape, x.stride()
    return x if (one == 1 or k <= 1) and (ld >= k or m <= 1) else x.contiguous()


class _Weights:
    """8-bit weights and what goes with them, checked once: pointers for the calls that follow.  The tensors are held
    here and not to be replaced."""

    def __init__(self, **named):
        self.tensors = [t for t, _, _ in named.values() if t is not None]
        self.dev = _device(self.tensors[0], next(iter(named)))
        for what, (t, shape, dtype) in named.items():
            setattr(self, what, _ptr(t, what, shape, self.dev, dtype))


class Q8Linear:
    """A linear layer in 8 bits: w int8 [N, K], one fp32 scale per output channel, optional fp16 bias.

    ``forward(x)`` cuts x [..., K] to 8 bits per token inside the call; ``forward_q8(q, s)`` takes tokens that are in
    8 bits already (block_norm, q8_quantize)."""

    def __init__(self, w, scale, bias=None):
        torch = _torch()
        n, k = self.out_features, self.in_features = w.shape
        self.w, self.scale, self.bias = q8_pad(w), scale, bias
        self._p = _Weights(w=(self.w, (n, q8_row_bytes(k)), torch.int8), scale=(scale, (n,), torch.float32),
                           bias=(bias, (n,), torch.float16))

    @classmethod
    def from_weight(cls, w, bias=None):
        """From a dense weight [N, K] (fp16, bf16 or fp32 on the device), cut to 8 bits per row."""
        q, s = q8_quantize(w)
        return cls(q[:, :w.shape[1]], s, bias)

    def forward(self, x, y_dtype=None):
        n, k, w = self.out_features, self.in_features, self._p
        rows = _tokens(x)
        p, ld, code, dev = _rows(rows, "x")
        if dev != w.dev or rows.shape[1] != k:
            raise ValueError("x must be [..., %d] on device %d, got %s on %s" % (k, w.dev, tuple(x.shape), x.device))
        m, stream = rows.shape[0], _stream(dev)
        y = rows.new_empty((m, n), dtype=y_dtype or x.dtype)
        nbytes = 0 if m == 1 and k <= ONE_MAX_K else q8_linear_workspace_bytes(m, n, k)
        ws, ws_p = _workspace(nbytes, rows)
        _launch(lib().vq_q8_linear, dev, m, n, k, p, code, ld, w.w, w.scale, w.bias, y.data_ptr(), _code(y.dtype), ws_p,
                nbytes, stream)
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], n)

    __call__ = forward

    def forward_q8(self, q, s, y_dtype=None):
        torch = _torch()
        n, k, w = self.out_features, self.in_features, self._p
        m, stream = q.shape[0], _stream(w.dev)
        y = q.new_empty((m, n), dtype=y_dtype or torch.bfloat16)
        nbytes = q8_gemm_workspace_bytes(m, n, k)
        ws, ws_p = _workspace(nbytes, q)
        _launch(lib().vq_q8_gemm, w.dev, m, n, k, _ptr(q, "q", (m, q8_row_bytes(k)), w.dev, torch.int8),
                _ptr(s, "s", (m,), w.dev, torch.float32), w.w, w.scale, w.bias, y.data_ptr(), _code(y.dtype), ws_p,
                nbytes, stream)
        return y


class Q8Experts:
    """An expert layer in 8 bits: w_in int8 [E, 2 I, D] (gate rows first), w_out int8 [E, D, I], fp32 channel scales
    s_in [E, 2 I] and s_out [E, D]."""

    def __init__(self, w_in, s_in, w_out, s_out):
        torch = _torch()
        e, d, i = w_out.shape
        # the padded rows of another width could be as long; rows that are padded already are taken as before
        if tuple(w_in.shape) not in ((e, 2 * i, d), (e, 2 * i, q8_row_bytes(d))):
            raise ValueError("w_in must be %s, got %s" % ([e, 2 * i, d], tuple(w_in.shape)))
        self.experts, self.features, self.inner = e, d, i
        self.w_in, self.s_in, self.w_out, self.s_out = q8_pad(w_in), s_in, q8_pad(w_out), s_out
        self._p = _Weights(w_in=(self.w_in, (e, 2 * i, q8_row_bytes(d)), torch.int8),
                           s_in=(s_in, (e, 2 * i), torch.float32),
                           w_out=(self.w_out, (e, d, q8_row_bytes(i)), torch.int8),
                           s_out=(s_out, (e, d), torch.float32))

    def forward(self, x, ids, p, y_dtype=None):
        """y [..., D] for x [..., D] and its tokens' expert ids (int32) and weights (fp32) [tokens, top]."""
        torch = _torch()
        e, d, i, w = self.experts, self.features, self.inner, self._p
        rows = _tokens(x)
        xp, ld, code, dev = _rows(rows, "x")
        if dev != w.dev or rows.shape[1] != d:
            raise ValueError("x must be [..., %d] on device %d, got %s on %s" % (d, w.dev, tuple(x.shape), x.device))
        if ids.dim() != 2:
            raise ValueError("ids must be [tokens, top], got %s" % (tuple(ids.shape),))
        t, top, stream = rows.shape[0], ids.shape[1], _stream(dev)
        y = rows.new_empty((t, d), dtype=y_dtype or x.dtype)
        nbytes = q8_experts_workspace_bytes(t, top, e, d, i)
        ws, ws_p = _workspace(nbytes, rows)
        _launch(lib().vq_q8_experts, dev, t, top, e, d, i, xp, code, ld, _ptr(ids, "ids", (t, top), dev, torch.int32),
                _ptr(p, "p", (t, top), dev, torch.float32), w.w_in, w.s_in, w.w_out, w.s_out, y.data_ptr(),
                _code(y.dtype), ws_p, nbytes, stream)
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], d)

    __call__ = forward
