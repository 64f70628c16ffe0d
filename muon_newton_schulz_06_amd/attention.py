"""The attention half of a block beside the layers: rotary positions,
differential attention, dropout with the residual's addition.

Functions named after the C entry points of ``include/muon_attention.h`` (the
binding marshals arguments only; every value is computed by the library's HIP
kernels, and without the built library the calls raise), and `torch.nn`
modules with autograd on top of them:

    muon_rotary / muon_rotary_grad                    Rotary
    muon_diff_attention / muon_diff_attention_grad    DiffAttention
    muon_dropout / muon_dropout_grad                  Dropout

Tensors of heads are (batch, tokens, heads, values), or (tokens, heads,
values), with any strides; inputs whose values are not contiguous
(stride(-1) != 1) are copied, outputs may not be so.  Otherwise the conventions
are those of the layers: float32 or bfloat16 on one CUDA/HIP device, work on the
current stream, or on ``stream``, a cached workspace unless one is passed; the
functions record nothing for autograd, the modules have a backward pass and
refuse forward-mode tangents.  Before a backward pass is captured into a graph,
drop the graphs that eager passes built of the same parameters: torch ties a
parameter to the stream of the first graph that is alive.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import _check, _raw_stream, _workspace, load
from .layers import _code, _device, _input, _on, _out, _ptr, _RMSNormFn, _rows, _same

__all__ = [
    "rotary_frequencies", "muon_rotary", "muon_rotary_grad", "muon_dropout", "muon_dropout_grad",
    "muon_diff_attention", "muon_diff_attention_grad", "diff_attention_saved_size",
    "diff_attention_workspace_size", "Rotary", "DiffAttention", "Dropout",
]

_i64x3 = ctypes.c_int64 * 3


class MuonRotary(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("tokens", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("rotated", ctypes.c_int64), ("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("position_stride", ctypes.c_int64), ("start", ctypes.c_int64),
                ("position_bytes", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class MuonRotaryHeads(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("in_strides", _i64x3), ("out_strides", _i64x3)]


_two_heads = MuonRotaryHeads * 2  # kept: ctypes makes the type anew, in 20 us, where nothing else holds it


class MuonDiffAttention(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("queries", ctypes.c_int64), ("keys", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("lam", ctypes.c_void_p),
                ("q_strides", _i64x3), ("k_strides", _i64x3), ("v_strides", _i64x3),
                ("offsets", ctypes.c_void_p), ("sequences", ctypes.c_int64), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MuonDiffAttentionGrads(ctypes.Structure):
    _fields_ = [("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
                ("dlam", ctypes.c_void_p), ("dq_strides", _i64x3), ("dk_strides", _i64x3), ("dv_strides", _i64x3)]


_bound = None


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    L = load()
    vp, i32, i64, u64, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                  ctypes.c_double, ctypes.c_size_t)
    psz = ctypes.POINTER(sz)
    pr, ph = ctypes.POINTER(MuonRotary), ctypes.POINTER(MuonRotaryHeads)
    pa, pg, ps = ctypes.POINTER(MuonDiffAttention), ctypes.POINTER(MuonDiffAttentionGrads), ctypes.POINTER(_i64x3)
    for name, args in {
        "muon_rotary": [pr, ph, i32, vp],
        "muon_rotary_grad": [pr, ph, i32, vp],
        "muon_dropout": [vp, i64, vp, i64, f64, u64, u64, vp, vp, i64, i64, i64, i32, vp],
        "muon_dropout_grad": [vp, i64, f64, u64, u64, vp, vp, i64, i64, i64, i32, vp],
        "muon_diff_attention": [pa, vp, ps, vp, sz, vp, sz, vp],
        "muon_diff_attention_grad": [pa, vp, ps, vp, ps, vp, sz, pg, vp, sz, vp],
        "muon_diff_attention_saved_size": [pa, psz],
        "muon_diff_attention_workspace_size": [pa, vp, ps, psz],
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i32
    _bound = L
    return L


def _heads(t, name):
    """(batch, tokens, heads, values) view of a 3-D or 4-D tensor."""
    if t.dim() == 3:
        return t.unsqueeze(0)
    if t.dim() != 4:
        raise ValueError(f"{name} must be (batch, tokens, heads, values) or (tokens, heads, values), got shape "
                         f"{tuple(t.shape)}")
    return t


def _contiguous_values(t):
    return t.shape[-1] <= 1 or t.stride(-1) == 1


def _input_heads(t, name):
    t = _heads(t, name)
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def _strides(t):
    b, n, h, _ = t.stride()
    return _i64x3(b, n, h)


def _like(t):
    """An uninitialised contiguous tensor of t's shape (the quickest way there)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _output(out, shape, dtype, dev, name):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {tuple(shape)}")
    _same(dev, dtype, **{name: out})
    if not _contiguous_values(out):
        raise ValueError(f"{name}: the values of a head must be contiguous (stride(-1) == 1)")
    return out


# ------------------------------------------------------------------- rotary

def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(freqs, scale): the dim/2 angles per position, base^(-2i/dim), as a
    float64 CPU tensor, and the factor that muon_rotary multiplies q and k
    with (1 but for "yarn").  For contexts ``factor`` times as long as the
    ``original_length`` a model was trained on:
      "linear": every frequency divided by factor (positions interpolated);
      "base":   base · factor^(dim/(dim-2)), which leaves the highest frequency
                and divides the lowest by factor;
      "yarn":   (Peng, Quesnelle, Fan, Shippole: YaRN, 2023) frequencies of at
                least ``fast`` turns over the original length are kept, of at
                most ``slow`` turns divided by factor, with a linear ramp over
                the index between; scale = 0.1·ln(factor) + 1."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and at least 2, got {dim}")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    i = torch.arange(dim // 2, dtype=torch.float64, device="cpu")
    if scaling == "base":
        if dim == 2:
            raise ValueError('scaling "base" needs dim > 2')
        base = base * factor ** (dim / (dim - 2))
    freqs = base ** (-2.0 * i / dim)
    if scaling in (None, "base"):
        return freqs, 1.0
    if scaling == "linear":
        return freqs / factor, 1.0
    if scaling != "yarn":
        raise ValueError(f'unknown scaling {scaling!r}; use None, "linear", "base" or "yarn"')
    if not original_length > 0 or not base > 1 or not 0 < slow <= fast:
        raise ValueError(f'scaling "yarn" needs original_length > 0, base > 1 and 0 < slow <= fast, got {original_length}, '
                         f"{base}, {slow} and {fast}")
    # the (fractional) index whose frequency makes n turns over the original length
    def index(n):
        return dim * math.log(original_length / (n * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), dim - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return freqs * (1.0 - ramp) + freqs / factor * ramp, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _rotary(entry, q, k, freqs, positions, start, interleaved, scale, q_out, k_out, stream):
    dev = _device(q, "q")
    code = _code(q, "q")
    if k is not None and (k.device != dev or k.dtype != q.dtype):
        _same(dev, q.dtype, k=k)
    if freqs.device != dev or freqs.dtype != torch.float64:
        _same(dev, torch.float64, freqs=freqs)
    if freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError(f"freqs must be a contiguous vector, got shape {tuple(freqs.shape)}")
    with _on(dev, stream):
        q4 = _input_heads(q, "q")
        batch, tokens, _, dim = q4.shape
        r = MuonRotary(batch, tokens, dim, 2 * freqs.numel(), _ptr(freqs), None, 0, int(start), 0,
                       int(bool(interleaved)), scale, code)
        if positions is not None:
            positions = _positions(r, positions, dev)
        arr = _two_heads()
        qo, kept = _turn(arr, 0, q, q4, q_out, "q")
        ko, n = None, 1
        if k is not None:
            k4 = _input_heads(k, "k")
            if k4.shape[0] != batch or k4.shape[1] != tokens or k4.shape[3] != dim or k.dim() != q.dim():
                raise ValueError(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}: only their heads may differ")
            (ko, kept2), n = _turn(arr, 1, k, k4, k_out, "k"), 2
        _check(entry(ctypes.byref(r), arr, n, _raw_stream(dev.index)))
    return qo, ko


def _positions(r, positions, dev):
    """Sets them in r; the tensor r then points into."""
    if positions.device != dev or positions.dtype not in (torch.int32, torch.int64):
        _same(dev, None, positions=positions)
        raise TypeError(f"positions have dtype {positions.dtype}; use int32 or int64")
    shape, tokens = tuple(positions.shape), r.tokens
    if shape not in ((tokens,), (1, tokens), (r.batch, tokens)):
        raise ValueError(f"positions have shape {shape}, expected ({tokens},) or ({r.batch}, {tokens})")
    if tokens > 1 and positions.stride(-1) != 1:
        positions = positions.contiguous()
    if len(shape) == 2 and shape[0] > 1:
        if 0 < positions.stride(0) < tokens:
            positions = positions.contiguous()
        r.position_stride = positions.stride(0)
    r.positions, r.position_bytes = _ptr(positions), positions.element_size()
    return positions


def _turn(arr, i, t, t4, out, name):
    """Sets tensor i of a call: (its output, what arr points into)."""
    o = _like(t) if out is None else _output(out, t.shape, t.dtype, t.device, name + "_out")
    o4 = o if o.dim() == 4 else o.unsqueeze(0)
    arr[i] = MuonRotaryHeads(_ptr(t4), _ptr(o4), t4.shape[2], _strides(t4), _strides(o4))
    return o, t4


def muon_rotary(q, k, freqs, positions=None, start: int = 0, interleaved: bool = False, scale: float = 1.0,
                q_out=None, k_out=None, stream=None):
    """(q', k'): the first 2·len(freqs) values of every head turned by
    position · freqs, times scale; the other values unchanged.  Pairs are
    (i, i + len(freqs)), or (2i, 2i + 1) with interleaved.  q, k (None: q
    alone): (batch, tokens, heads, dim) or (tokens, heads, dim); freqs:
    float64; positions: int32 or int64, (tokens,) or (batch, tokens), by
    default start, start + 1, …  q_out and k_out may be q and k (in place)."""
    return _rotary(_lib().muon_rotary, q, k, freqs, positions, start, interleaved, scale, q_out, k_out, stream)


def muon_rotary_grad(dq, dk, freqs, positions=None, start: int = 0, interleaved: bool = False, scale: float = 1.0,
                     q_out=None, k_out=None, stream=None):
    """Gradients of muon_rotary's q and k from those of its results: the
    rotation by the opposite angles.  Arguments as there."""
    return _rotary(_lib().muon_rotary_grad, dq, dk, freqs, positions, start, interleaved, scale, q_out, k_out,
                   stream)


# ------------------------------------------------------------------ dropout

_U64 = (1 << 64) - 1


def _offset(offset, dev):
    """(host value, device tensor or None)"""
    if not torch.is_tensor(offset):
        return int(offset) & _U64, None
    _same(dev, torch.int64, offset=offset)
    if offset.numel() != 1:
        raise ValueError("offset must be a number or an int64 tensor of one element")
    return 0, offset


def muon_dropout(x, p: float, seed: int, offset=0, residual=None, out=None, stream=None):
    """residual + x/(1 - p) where an element is kept, residual (or 0)
    elsewhere.  An element's random word depends on its index in x, seed and
    offset alone, so nothing has to be kept for the backward pass.  offset: a
    number, or an int64 tensor of one element on x's device, read when the
    kernel runs (so that a replayed graph can draw anew).  out may be x or
    residual (in place)."""
    L = _lib()
    dev = _device(x, "x")
    code = _code(x, "x")
    _same(dev, x.dtype, residual=residual)
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
    host, tensor = _offset(offset, dev)
    with _on(dev, stream):
        x2, ldx = _input(x, "x")
        r2, ldr = _input(residual, "residual") if residual is not None else (None, 0)
        y = _like(x) if out is None else _out(out, x.shape, x.dtype, dev, "out")
        y2, ldy = _rows(y, "out")
        if y.numel():
            _check(L.muon_dropout(_ptr(x2), ldx, _ptr(r2), ldr, p, int(seed) & _U64, host, _ptr(tensor), _ptr(y2), ldy,
                                  x2.shape[0], x2.shape[1], code, _raw_stream(dev.index)))
    return y


def muon_dropout_grad(dy, p: float, seed: int, offset=0, out=None, stream=None):
    """Gradient of muon_dropout's x from dy (its residual's gradient is dy),
    with the arguments of that call.  out may be dy (in place)."""
    L = _lib()
    dev = _device(dy, "dy")
    code = _code(dy, "dy")
    host, tensor = _offset(offset, dev)
    with _on(dev, stream):
        d2, ldd = _input(dy, "dy")
        y = _like(dy) if out is None else _out(out, dy.shape, dy.dtype, dev, "out")
        y2, ldy = _rows(y, "out")
        if y.numel():
            _check(L.muon_dropout_grad(_ptr(d2), ldd, p, int(seed) & _U64, host, _ptr(tensor), _ptr(y2), ldy,
                                       d2.shape[0], d2.shape[1], code, _raw_stream(dev.index)))
    return y


# --------------------------------------------------- differential attention

def _attention(q, k, v, lam, causal, scale, offsets):
    """The call's descriptor, and the tensors it points into."""
    code = _code(q, "q")
    dev = q.device
    _same(dev, q.dtype, k=k, v=v)
    _same(dev, torch.float32, lam=lam)
    if not q.dim() == k.dim() == v.dim():
        raise ValueError("q, k and v must have the same number of dimensions")
    if offsets is not None and q.dim() != 3:
        raise ValueError("a packed batch (offsets) takes tensors of (tokens, heads, values)")
    q4, k4, v4 = (_input_heads(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    batch, queries, qh, dim = q4.shape
    keys, kh = k4.shape[1:3]
    if qh < 2 or qh % 2 or kh < 2 or kh % 2:
        raise ValueError(f"q and k must have two heads per map pair, got {qh} and {kh}")
    if k4.shape[0] != batch or k4.shape[3] != dim:
        raise ValueError(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
    if tuple(v4.shape) != (batch, keys, kh // 2, 2 * dim):
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {(batch, keys, kh // 2, 2 * dim)[4 - v.dim():]}")
    if tuple(lam.shape) != (qh // 2,):
        raise ValueError(f"lam has shape {tuple(lam.shape)}, expected ({qh // 2},)")
    lam = lam.contiguous()
    f = MuonDiffAttention(batch, queries, keys, qh // 2, kh // 2, dim, _ptr(q4), _ptr(k4), _ptr(v4), _ptr(lam),
                          _strides(q4), _strides(k4), _strides(v4), None, 0,
                          max(dim, 1) ** -0.5 if scale is None else scale, int(bool(causal)), code)
    if offsets is not None:
        _same(dev, torch.int32, offsets=offsets)
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets must be a vector of one more element than sequences, two at least")
        offsets = offsets.contiguous()
        f.offsets, f.sequences = _ptr(offsets), offsets.numel() - 1
    return f, (q4, k4, v4, lam, offsets)


def _attention_sizes(batch, queries, keys, heads, kv_heads, dim, dtype, sequences):
    code = _code(torch.empty(0, dtype=dtype), "dtype")
    z = _i64x3(1, 1, 1)  # off every alignment: room for copies
    return MuonDiffAttention(int(batch), int(queries), int(keys), int(heads), int(kv_heads), int(dim), 1, 1, 1, None,
                             z, z, z, None, int(sequences), 1.0, 0, code)


def diff_attention_saved_size(batch, queries, keys, heads, kv_heads, dim, dtype=torch.bfloat16) -> int:
    """Bytes muon_diff_attention(save=True) keeps for the backward pass."""
    f, n = _attention_sizes(batch, queries, keys, heads, kv_heads, dim, dtype, 0), ctypes.c_size_t(0)
    _check(_lib().muon_diff_attention_saved_size(ctypes.byref(f), ctypes.byref(n)))
    return n.value


def diff_attention_workspace_size(batch, queries, keys, heads, kv_heads, dim, dtype=torch.bfloat16,
                                  grad: bool = False, sequences: int = 0) -> int:
    """Workspace bytes of muon_diff_attention, or of its gradient, enough for
    tensors of any strides; sequences: those of a packed batch."""
    f, n = _attention_sizes(batch, queries, keys, heads, kv_heads, dim, dtype, sequences), ctypes.c_size_t(0)
    _check(_lib().muon_diff_attention_workspace_size(ctypes.byref(f), 1 if grad else None, _i64x3(1, 1, 1),
                                                     ctypes.byref(n)))
    return n.value


def muon_diff_attention(q, k, v, lam, causal: bool = True, scale: float | None = None, offsets=None,
                        save: bool = False, out=None, workspace=None, stream=None):
    """(softmax(scale·q₁·k₁ᵀ) − lam·softmax(scale·q₂·k₂ᵀ))·v per head, where
    q₁, q₂ are the query heads 2h and 2h + 1 and k₁, k₂ the key heads 2g and
    2g + 1 of the head's group g.  q: (batch, queries, 2·heads, dim), k:
    (batch, keys, 2·kv_heads, dim), v: (batch, keys, kv_heads, 2·dim), lam:
    float32 (heads,); without the batch dimension, one sequence, or with
    ``offsets`` (int32, one more than sequences) a packed batch of them.
    causal: the last query sees the last key.  scale: by default dim^-0.5.
    Returns out (…, queries, heads, 2·dim), or (out, saved) with save: an opaque
    uint8 tensor that muon_diff_attention_grad takes."""
    L = _lib()
    dev = _device(q, "q")
    with _on(dev, stream):
        f, kept = _attention(q, k, v, lam, causal, scale, offsets)
        shape = (f.batch, f.queries, f.heads, 2 * f.dim)
        y = _output(out, shape[4 - q.dim():], q.dtype, dev, "out")
        n = ctypes.c_size_t(0)
        saved, nsaved = None, 0
        if save:
            _check(L.muon_diff_attention_saved_size(ctypes.byref(f), ctypes.byref(n)))
            nsaved = n.value
            saved = torch.empty(nsaved, dtype=torch.uint8, device=dev)
        _check(L.muon_diff_attention_workspace_size(ctypes.byref(f), None, None, ctypes.byref(n)))
        with _workspace(n.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_diff_attention(ctypes.byref(f), _ptr(y), _strides(_heads(y, "out")), _ptr(saved), nsaved,
                                         _ptr(ws), nbytes, _raw_stream(dev.index)))
    return (y, saved) if save else y


def muon_diff_attention_grad(dout, q, k, v, lam, out, saved, causal: bool = True, scale: float | None = None,
                             offsets=None, want_dq: bool = True, want_dkv: bool = True, want_dlam: bool = True,
                             workspace=None, stream=None):
    """(dq, dk, dv, dlam) of muon_diff_attention from dout, its result ``out``
    and ``saved``, with the arguments of that call; None for those not
    wanted."""
    L = _lib()
    dev = _device(q, "q")
    _same(dev, q.dtype, dout=dout, out=out)
    _same(dev, torch.uint8, saved=saved)
    if not saved.is_contiguous():
        raise ValueError("saved must be contiguous, as muon_diff_attention returned it")
    with _on(dev, stream):
        f, kept = _attention(q, k, v, lam, causal, scale, offsets)
        shape = (f.batch, f.queries, f.heads, 2 * f.dim)[4 - q.dim():]
        for name, t in (("dout", dout), ("out", out)):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        d4, o4 = _input_heads(dout, "dout"), _input_heads(out, "out")
        grads = [_like(t) if want else None
                 for t, want in ((q, want_dq), (k, want_dkv), (v, want_dkv))]
        dlam = torch.empty(f.heads, dtype=torch.float32, device=dev) if want_dlam else None
        none = _i64x3(0, 0, 0)
        g = MuonDiffAttentionGrads(*(_ptr(t) for t in grads), _ptr(dlam),
                                   *(none if t is None else _strides(_heads(t, "gradient")) for t in grads))
        n, ds = ctypes.c_size_t(0), _strides(d4)
        # an empty dout has no address, but the size is that of the backward pass
        _check(L.muon_diff_attention_workspace_size(ctypes.byref(f), _ptr(d4) or 16, ds, ctypes.byref(n)))
        with _workspace(n.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_diff_attention_grad(ctypes.byref(f), _ptr(d4), ds, _ptr(o4), _strides(o4), _ptr(saved),
                                              saved.numel(), ctypes.byref(g), _ptr(ws), nbytes,
                                              _raw_stream(dev.index)))
    return (*grads, dlam)


# ------------------------------------------------------------------ autograd

class _RotaryFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, freqs, positions, start, interleaved, scale):
        ctx.save_for_backward(freqs, positions)
        ctx.how = (start, interleaved, scale)
        ctx.set_materialize_grads(False)
        return muon_rotary(q, k, freqs, positions, start, interleaved, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        freqs, positions = ctx.saved_tensors
        if dq is None or dk is None:  # one of the two alone
            one = dk if dq is None else dq
            if one is not None:
                one, _ = muon_rotary_grad(one, None, freqs, positions, *ctx.how)
            dq, dk = (None, one) if dq is None else (one, None)
        else:
            dq, dk = muon_rotary_grad(dq, dk, freqs, positions, *ctx.how)
        return dq, dk, None, None, None, None, None


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.how = (p, seed)
        ctx.save_for_backward(offset)
        return muon_dropout(x, p, seed, offset, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (offset,) = ctx.saved_tensors
        dx = muon_dropout_grad(dy, *ctx.how, offset) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


class _DiffAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, causal, scale, offsets, save):
        ctx.how = (causal, scale)
        if not save:  # no backward pass will come
            return muon_diff_attention(q, k, v, lam, causal, scale, offsets)
        out, saved = muon_diff_attention(q, k, v, lam, causal, scale, offsets, save=True)
        ctx.save_for_backward(q, k, v, lam, out, saved, offsets)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, lam, out, saved, offsets = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = muon_diff_attention_grad(dout, q, k, v, lam, out, saved, *ctx.how, offsets, want_dq=need[0],
                                         want_dkv=need[1] or need[2], want_dlam=need[3])
        return (*grads, None, None, None, None)


class Rotary(torch.nn.Module):
    """Rotates queries and keys by their positions.  rotated: the values of a
    head that take part (by default all ``dim``); the scalings for long contexts
    are rotary_frequencies'.  The first call on a device copies the frequencies
    there, so it cannot be one that is captured into a graph."""

    def __init__(self, dim: int, rotated: int | None = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: str | None = None, factor: float = 1.0, original_length: int = 0):
        super().__init__()
        rotated = dim if rotated is None else rotated
        if rotated > dim:
            raise ValueError(f"rotated ({rotated}) above dim ({dim})")
        with torch.inference_mode(False):
            self.freqs, self.scale = rotary_frequencies(rotated, base, scaling, factor, original_length)
        self.dim, self.interleaved = dim, bool(interleaved)
        self._here = {}  # the frequencies per device: fp64 whatever dtype the module is cast to

    def forward(self, q, k=None, positions=None, start: int = 0):
        """(q', k') of q and k (batch, tokens, heads, dim), q' alone without k."""
        if q.shape[-1] != self.dim:
            raise ValueError(f"heads of {q.shape[-1]} values, expected {self.dim}")
        freqs = self._here.get(q.device)
        if freqs is None:
            with torch.inference_mode(False):  # (a later backward pass may save them)
                freqs = self._here[q.device] = self.freqs.to(q.device, copy=True)
        q, k = _RotaryFn.apply(q, k, freqs, positions, start, self.interleaved, self.scale)
        return q if k is None else (q, k)


class Dropout(torch.nn.Module):
    """residual + dropout(x): each call of the training mode draws anew, from
    the seed and a counter of the calls on the device (so that replays of a
    captured graph draw anew too).  In evaluation mode, or with p = 0, the
    addition alone.

    seed: by default drawn from torch's CPU generator; it is part of the state.
    Modules (and ranks) with equal seeds drop the same elements.  The counter
    goes by calls: a forward pass repeated to save memory would draw again."""

    def __init__(self, p: float, seed: int | None = None, device=None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be in [0, 1], got {p}")
        self.p, self.seed = float(p), int(torch.randint(1 << 62, (), device="cpu")) if seed is None else int(seed)
        self.register_buffer("calls", torch.zeros(1, dtype=torch.int64, device=device))

    def get_extra_state(self):
        return self.seed

    def set_extra_state(self, seed):
        self.seed = int(seed)

    def forward(self, x, residual=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else x + residual
        offset = self.calls.clone()
        self.calls.add_(1)
        return _DropoutFn.apply(x, residual, self.p, self.seed, offset)


class DiffAttention(torch.nn.Module):
    """Differential attention of projected (and rotated) queries, keys and
    values, with its learned λ and the norm of each head's result:

        λ = exp(λ_q1·λ_k1) − exp(λ_q2·λ_k2) + λ_init,
        (1 − λ_init) · RMSNorm(attention(q, k, v, λ)) over the 2·dim values of a
        head, one weight vector for all heads.

    forward(q, k, v, offsets=None): (batch, tokens, 2·heads, dim), (batch, tokens,
    2·kv_heads, dim), (batch, tokens, kv_heads, 2·dim) to (batch, tokens, heads,
    2·dim); a packed batch without the batch dimension and with offsets.  The norm
    takes up to 2^24 rows: batch · tokens · heads."""

    def __init__(self, heads: int, dim: int, kv_heads: int | None = None, lambda_init: float = 0.8,
                 causal: bool = True, eps: float = 1e-5, device=None, dtype=None):
        super().__init__()
        self.heads, self.kv_heads, self.dim = heads, heads if kv_heads is None else kv_heads, dim
        if heads < 1 or self.kv_heads < 1 or heads % self.kv_heads:
            raise ValueError(f"kv_heads ({self.kv_heads}) must divide heads ({heads})")
        self.lambda_init, self.causal, self.eps = float(lambda_init), bool(causal), float(eps)
        for name in ("lambda_q1", "lambda_k1", "lambda_q2", "lambda_k2"):
            setattr(self, name, torch.nn.Parameter(torch.empty(dim, device=device, dtype=torch.float32).normal_(std=0.1)))
        self.weight = torch.nn.Parameter(torch.ones(2 * dim, device=device, dtype=dtype))

    def lam(self):
        """λ, one value per head (the same for all), float32."""
        one = (self.lambda_q1.float() * self.lambda_k1.float()).sum().exp()
        two = (self.lambda_q2.float() * self.lambda_k2.float()).sum().exp()
        return (one - two + self.lambda_init).expand(self.heads)

    def forward(self, q, k, v, offsets=None):
        if q.shape[-2:] != (2 * self.heads, self.dim) or k.shape[-2:] != (2 * self.kv_heads, self.dim):
            raise ValueError(f"q and k have shapes {tuple(q.shape)} and {tuple(k.shape)}, expected heads of "
                             f"({2 * self.heads}, {self.dim}) and ({2 * self.kv_heads}, {self.dim})")
        lam = self.lam()
        save = torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v, lam))
        out = _DiffAttentionFn.apply(q, k, v, lam, self.causal, None, offsets, save)
        return _RMSNormFn.apply(out, self.weight * (1.0 - self.lambda_init), None, self.eps)
