"""The layers whose gradients the Muon step consumes: embedding lookup, RMS
norm with the residual's addition, gated feed-forward block.

Functions named after the C entry points of ``include/muon_layers.h`` (the
binding marshals arguments only; every value is computed by the library's HIP
kernels, and without the built library the calls raise), and `torch.nn`
modules with autograd on top of them:

    muon_embedding / muon_embedding_grad        Embedding
    muon_rms_norm / muon_rms_norm_grad          RMSNorm
    muon_gated_ffn / muon_gated_ffn_grad        GatedFFN

The functions record nothing for autograd (and drop tangents); the modules
have a backward pass, and refuse forward-mode tangents.

Tensors are float32 or bfloat16 on one CUDA/HIP device.  Leading dimensions
are flattened to rows, which may have any stride; inputs whose rows are not
contiguous (stride(-1) != 1), or overlap, are copied, weights and outputs may
not have such rows.  Work runs on the current stream, or on ``stream`` (outputs are
then allocated for that stream; the caller orders the inputs' writes before
it).  A workspace is cached per device and stream unless one is passed.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import MUON_DTYPE_BF16, MUON_DTYPE_F32, _check, _raw_stream, _workspace, load

__all__ = [
    "ACTIVATIONS", "muon_embedding", "muon_embedding_grad", "muon_rms_norm", "muon_rms_norm_grad",
    "muon_gated_ffn", "muon_gated_ffn_grad", "gated_ffn_saved_size", "gated_ffn_workspace_size",
    "Embedding", "RMSNorm", "GatedFFN",
]

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class MuonFfn(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("model", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("ld_gate", ctypes.c_int64), ("ld_up", ctypes.c_int64), ("ld_down", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class MuonFfnGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dw_gate", ctypes.c_void_p), ("dw_up", ctypes.c_void_p),
                ("dw_down", ctypes.c_void_p), ("ld_dx", ctypes.c_int64), ("ld_gate", ctypes.c_int64),
                ("ld_up", ctypes.c_int64), ("ld_down", ctypes.c_int64), ("grad_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32)]


_bound = None


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    L = load()
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    psz = ctypes.POINTER(sz)
    pf, pg = ctypes.POINTER(MuonFfn), ctypes.POINTER(MuonFfnGrads)
    for name, args in {
        "muon_embedding": [vp, i32, i64, vp, i64, i64, i64, f32, vp, i64, i32, vp],
        "muon_embedding_grad": [vp, i64, vp, i32, i64, i64, i64, f32, vp, i64, i32, i32, i32, vp, sz, vp],
        "muon_embedding_grad_workspace_size": [i64, i64, i64, psz],
        "muon_rms_norm": [vp, i64, vp, i64, vp, i32, f32, vp, i64, vp, i64, vp, i64, i64, i32, vp],
        "muon_rms_norm_grad": [vp, i64, vp, i64, vp, i32, vp, vp, i64, vp, i64, vp, i32, i64, i64, i32,
                               vp, sz, vp],
        "muon_rms_norm_grad_workspace_size": [i64, i64, psz],
        "muon_gated_ffn": [pf, vp, i64, vp, i64, vp, sz, vp, sz, vp],
        "muon_gated_ffn_grad": [pf, vp, i64, vp, i64, vp, sz, pg, vp, sz, vp],
        "muon_gated_ffn_saved_size": [pf, psz],
        "muon_gated_ffn_workspace_size": [pf, i32, psz],
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i32
    _bound = L
    return L


_CODES = {torch.float32: MUON_DTYPE_F32, torch.bfloat16: MUON_DTYPE_BF16}


def _code(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} has dtype {t.dtype}; use float32 or bfloat16")
    return c


def _same(dev, dt, **tensors):
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}: all tensors must be on one device")
        if dt is not None and t.dtype != dt:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")


def _device(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA/HIP device, got {t.device}")
    return t.device


def _flat(t, name):
    """The tensor's rows, leading dimensions flattened."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    return t.reshape(-1, t.shape[-1]) if t.numel() else t.new_empty((math.prod(t.shape[:-1]), t.shape[-1]))


def _ld(t):
    """Row stride of a 2-D tensor, None if its rows are not contiguous or
    overlap."""
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1 and rows > 0:
        return None
    ld = s0 if rows > 1 else cols
    return ld if ld >= cols else None


def _rows(t, name):
    """(2-D view, row stride) of a weight or an output."""
    t = _flat(t, name)
    ld = _ld(t)
    if ld is None:
        raise ValueError(f"{name}: rows must be contiguous (stride(-1) == 1) and not overlap")
    return t, ld


def _input(t, name):
    """(2-D tensor, row stride) of an input: its view, or a copy where its
    rows are not contiguous (a transposed or broadcast tensor, as autograd may
    hand over)."""
    t = _flat(t, name)
    ld = _ld(t)
    return (t, ld) if ld is not None else (t.contiguous(), t.shape[1])


def _matrix(t, name, rows, cols):
    """Row stride of a 2-D tensor of the given shape."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({rows}, {cols})")
    return _rows(t, name)[1]


def _vector(t, name, n):
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values, got shape {tuple(t.shape)}")


class _On:
    """The device guard and stream of a call that cannot run as it is: the
    given stream is made current (so that outputs are allocated for it), and
    so is the tensors' device."""
    __slots__ = ("guard",)

    def __init__(self, dev, stream):
        self.guard = [torch.cuda.device(dev)]
        if stream is not None:
            self.guard.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guard:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guard):
            g.__exit__(*exc)
        return False


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    if stream is None and dev.index == torch.cuda.current_device():
        return _HERE
    return _On(dev, stream)


def _out(out, shape, dtype, dev, name):
    if out is None:
        return _empty(shape, dtype, dev)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {tuple(shape)}")
    _same(dev, dtype, **{name: out})
    if out.dim() != 2 and not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous (or 2-D)")
    return out


def _empty(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev)


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() else None


def _ids(ids):
    if ids.dtype == torch.int64:
        return ids.contiguous(), 8
    if ids.dtype == torch.int32:
        return ids.contiguous(), 4
    raise TypeError(f"ids have dtype {ids.dtype}; use int32 or int64")


# ---------------------------------------------------------------- embedding

def muon_embedding(ids, weight, scale: float = 1.0, out=None, stream=None):
    """out[..., :] = scale · weight[ids[...]]; a row of zeros where an id is
    outside [0, vocab) (padding).  ids: int32 or int64, any shape; weight:
    vocab × dim.  Returns a tensor of shape ids.shape + (dim,)."""
    L = _lib()
    dev = _device(weight, "weight")
    code = _code(weight, "weight")
    if weight.dim() != 2:
        raise ValueError(f"weight must be 2-D, got shape {tuple(weight.shape)}")
    _same(dev, None, ids=ids)
    vocab, dim = weight.shape
    _, ldw = _rows(weight, "weight")
    with _on(dev, stream):
        ids, nb = _ids(ids)
        out = _out(out, (*ids.shape, dim), weight.dtype, dev, "out")
        o, ldo = _rows(out, "out")
        _check(L.muon_embedding(_ptr(ids), nb, ids.numel(), _ptr(weight), ldw, vocab, dim, scale, _ptr(o),
                                ldo, code, _raw_stream(dev.index)))
    return out


def muon_embedding_grad(dy, ids, vocab: int, scale: float = 1.0, out=None, dtype=None,
                        accumulate: bool = False, workspace=None, stream=None):
    """Gradient of muon_embedding's weight: out[v] = scale · Σ dy over the
    tokens with id v (zero rows for absent ids), or, with accumulate, that sum
    added to ``out``.  dy: ids.shape + (dim,); out: vocab × dim, float32 or
    bfloat16 (allocated in ``dtype``, by default dy's, if None)."""
    L = _lib()
    dev = _device(dy, "dy")
    code = _code(dy, "dy")
    _same(dev, None, ids=ids)
    if tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"dy has shape {tuple(dy.shape)}, ids {tuple(ids.shape)}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dim, tokens = dy.shape[-1], ids.numel()
    vocab = int(vocab)
    with _on(dev, stream):
        ids, nb = _ids(ids)
        d, ldy = _input(dy, "dy")
        if out is None:
            out = torch.empty((vocab, dim), dtype=dtype or dy.dtype, device=dev)
        ldo = _matrix(out, "out", vocab, dim)
        _same(dev, dtype, out=out)
        need = ctypes.c_size_t(0)
        _check(L.muon_embedding_grad_workspace_size(tokens, vocab, dim, ctypes.byref(need)))
        with _workspace(need.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_embedding_grad(_ptr(d), ldy, _ptr(ids), nb, tokens, vocab, dim, scale, _ptr(out), ldo,
                                         code, _code(out, "out"), int(bool(accumulate)), _ptr(ws), nbytes,
                                         _raw_stream(dev.index)))
    return out


# ----------------------------------------------------------------- RMS norm

def muon_rms_norm(x, weight, residual=None, eps: float = 1e-6, out=None, sum_out=None, stream=None):
    """(y, s, rstd) of s = x + residual, rstd = 1/√(mean(s²) + eps) over the
    last dimension, y = s·rstd·weight (from s before it is rounded to x's
    dtype).  Without residual s is x itself.  weight: float32 or bfloat16;
    rstd: float32, of shape x.shape[:-1].  out and sum_out may be x or
    residual (in place)."""
    L = _lib()
    dev = _device(x, "x")
    code = _code(x, "x")
    _same(dev, x.dtype, residual=residual)
    _same(dev, None, weight=weight)
    dim = x.shape[-1]
    _vector(weight, "weight", dim)
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs residual")
    with _on(dev, stream):
        x2, ldx = _input(x, "x")
        r2, ldr = _input(residual, "residual") if residual is not None else (None, 0)
        y = _out(out, x.shape, x.dtype, dev, "out")
        y2, ldy = _rows(y, "out")
        s, s2, lds = x, None, 0
        if residual is not None:
            s = _out(sum_out, x.shape, x.dtype, dev, "sum_out")
            s2, lds = _rows(s, "sum_out")
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        _check(L.muon_rms_norm(_ptr(x2), ldx, _ptr(r2), ldr, _ptr(weight), _code(weight, "weight"), eps,
                               _ptr(y2), ldy, _ptr(s2), lds, _ptr(rstd), x2.shape[0], dim, code, _raw_stream(dev.index)))
    return y, s, rstd


def muon_rms_norm_grad(dy, s, weight, rstd, dsum=None, out=None, dweight=None, accumulate: bool = False,
                       want_dweight: bool = True, workspace=None, stream=None):
    """(dx, dweight) of muon_rms_norm: dx is the gradient of x and of residual
    alike, including ``dsum``, the gradient that reaches s by other ways.
    dweight has weight's dtype (added to the given one with accumulate; None
    with want_dweight false).  out may be dy or dsum (in place)."""
    L = _lib()
    dev = _device(dy, "dy")
    code = _code(dy, "dy")
    _same(dev, dy.dtype, s=s, dsum=dsum)
    _same(dev, torch.float32, rstd=rstd)
    _same(dev, None, weight=weight)
    dim = dy.shape[-1]
    _vector(weight, "weight", dim)
    for name, t in (("s", s), ("dsum", dsum)):
        if t is not None and t.shape != dy.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, dy {tuple(dy.shape)}")
    if accumulate and dweight is None:
        raise ValueError("accumulate needs dweight")
    with _on(dev, stream):
        dy2, ldy = _input(dy, "dy")
        s2, lds = _input(s, "s")
        d2, ldd = _input(dsum, "dsum") if dsum is not None else (None, 0)
        tokens = dy2.shape[0]
        if rstd.numel() != tokens or not rstd.is_contiguous():
            raise ValueError(f"rstd must hold {tokens} contiguous values, got shape {tuple(rstd.shape)}")
        dx = _out(out, dy.shape, dy.dtype, dev, "out")
        dx2, ldx = _rows(dx, "out")
        need = ctypes.c_size_t(0)
        if want_dweight:
            dweight = _out(dweight, (dim,), weight.dtype, dev, "dweight")
            _check(L.muon_rms_norm_grad_workspace_size(tokens, dim, ctypes.byref(need)))
        else:
            dweight = None
        with _workspace(need.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_rms_norm_grad(_ptr(dy2), ldy, _ptr(s2), lds, _ptr(weight), _code(weight, "weight"),
                                        _ptr(rstd), _ptr(d2), ldd, _ptr(dx2), ldx, _ptr(dweight),
                                        int(bool(accumulate)), tokens, dim, code, _ptr(ws), nbytes,
                                        _raw_stream(dev.index)))
    return dx, dweight


# -------------------------------------------------- gated feed-forward block

def _ffn(x, w_gate, w_up, w_down, activation):
    """The call's sizes and weights, with x as rows."""
    code = _code(x, "x")
    _same(x.device, x.dtype, w_gate=w_gate, w_up=w_up, w_down=w_down)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}; use one of {sorted(ACTIVATIONS)}")
    x2, ldx = _input(x, "x")
    tokens, model = x2.shape
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be 2-D, got shape {tuple(w_gate.shape)}")
    hidden = w_gate.shape[0]
    f = MuonFfn(tokens, model, hidden, _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                _matrix(w_gate, "w_gate", hidden, model), _matrix(w_up, "w_up", hidden, model),
                _matrix(w_down, "w_down", model, hidden), code, act)
    return f, x2, ldx


def _ffn_sizes(tokens, model, hidden, dtype, weights=None):
    """The call's sizes alone; without weights as if those lay off every
    alignment, which takes the most workspace."""
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    tokens, model, hidden = int(tokens), int(model), int(hidden)
    if weights is None:
        return MuonFfn(tokens, model, hidden, 1, 1, 1, model, model, hidden, code, 0)
    w_gate, w_up, w_down = weights
    _same(w_gate.device, dtype, w_gate=w_gate, w_up=w_up, w_down=w_down)
    return MuonFfn(tokens, model, hidden, _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                   _matrix(w_gate, "w_gate", hidden, model), _matrix(w_up, "w_up", hidden, model),
                   _matrix(w_down, "w_down", model, hidden), code, 0)


def gated_ffn_saved_size(tokens, model, hidden, dtype=torch.bfloat16) -> int:
    """Bytes muon_gated_ffn(save=True) keeps for the backward pass."""
    f, n = _ffn_sizes(tokens, model, hidden, dtype), ctypes.c_size_t(0)
    _check(_lib().muon_gated_ffn_saved_size(ctypes.byref(f), ctypes.byref(n)))
    return n.value


def gated_ffn_workspace_size(tokens, model, hidden, dtype=torch.bfloat16, grad: bool = False,
                             weights=None) -> int:
    """Workspace bytes of muon_gated_ffn, or of muon_gated_ffn_grad: for the
    given weights (w_gate, w_up, w_down), or enough for any.  bfloat16 weights
    whose rows are not whole aligned 16-byte chunks need room for a copy."""
    f, n = _ffn_sizes(tokens, model, hidden, dtype, weights), ctypes.c_size_t(0)
    _check(_lib().muon_gated_ffn_workspace_size(ctypes.byref(f), int(bool(grad)), ctypes.byref(n)))
    return n.value


def muon_gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu", save: bool = False, out=None,
                   workspace=None, stream=None):
    """y = (act(x·w_gateᵀ) · (x·w_upᵀ))·w_downᵀ over the last dimension of x.
    w_gate, w_up: hidden × model; w_down: model × hidden; all of x's dtype.
    Returns y, or (y, saved) with save: an opaque uint8 tensor that
    muon_gated_ffn_grad takes."""
    L = _lib()
    dev = _device(x, "x")
    with _on(dev, stream):
        f, x2, ldx = _ffn(x, w_gate, w_up, w_down, activation)
        y = _out(out, x.shape, x.dtype, dev, "out")
        y2, ldy = _rows(y, "out")
        n = ctypes.c_size_t(0)
        saved, nsaved = None, 0
        if save:
            _check(L.muon_gated_ffn_saved_size(ctypes.byref(f), ctypes.byref(n)))
            nsaved = n.value
            saved = torch.empty(nsaved, dtype=torch.uint8, device=dev)
        _check(L.muon_gated_ffn_workspace_size(ctypes.byref(f), 0, ctypes.byref(n)))
        with _workspace(n.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_gated_ffn(ctypes.byref(f), _ptr(x2), ldx, _ptr(y2), ldy, _ptr(saved), nsaved,
                                    _ptr(ws), nbytes, _raw_stream(dev.index)))
    return (y, saved) if save else y


def muon_gated_ffn_grad(dy, x, w_gate, w_up, w_down, saved, want_dx: bool = True, grads=None,
                        grad_dtype=None, accumulate: bool = False, want_dweights: bool = True,
                        workspace=None, stream=None):
    """(dx, dw_gate, dw_up, dw_down) of muon_gated_ffn from dy and ``saved``.
    The weight gradients go to ``grads`` (three tensors of the weights' shapes,
    float32 or bfloat16; added to them with accumulate) or are allocated in
    grad_dtype (by default the weights')."""
    L = _lib()
    dev = _device(x, "x")
    _same(dev, x.dtype, dy=dy)
    _same(dev, torch.uint8, saved=saved)
    if not saved.is_contiguous():
        raise ValueError("saved must be contiguous, as muon_gated_ffn returned it")
    if dy.shape != x.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, x {tuple(x.shape)}")
    if accumulate and grads is None:
        raise ValueError("accumulate needs grads")
    with _on(dev, stream):
        f, x2, ldx = _ffn(x, w_gate, w_up, w_down, "silu")
        dy2, ldy = _input(dy, "dy")
        dx, dx2, lddx = None, None, 0
        if want_dx:
            dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
            dx2, lddx = _rows(dx, "dx")
        g = MuonFfnGrads(_ptr(dx2), None, None, None, lddx, 0, 0, 0, 0, int(bool(accumulate)))
        out = (None, None, None)
        if want_dweights:
            if grads is None:
                dt = grad_dtype or x.dtype
                grads = [torch.empty(w.shape, dtype=dt, device=dev) for w in (w_gate, w_up, w_down)]
            out = tuple(grads)
            if len(out) != 3:
                raise ValueError("grads must be three tensors")
            _same(dev, grad_dtype or out[0].dtype, dw_gate=out[0], dw_up=out[1], dw_down=out[2])
            g.ld_gate = _matrix(out[0], "dw_gate", f.hidden, f.model)
            g.ld_up = _matrix(out[1], "dw_up", f.hidden, f.model)
            g.ld_down = _matrix(out[2], "dw_down", f.model, f.hidden)
            g.dw_gate, g.dw_up, g.dw_down = (_ptr(t) for t in out)
            g.grad_dtype = _code(out[0], "dw_gate")
        n = ctypes.c_size_t(0)
        _check(L.muon_gated_ffn_workspace_size(ctypes.byref(f), 1, ctypes.byref(n)))
        with _workspace(n.value, dev, workspace, stream) as (ws, nbytes):
            _check(L.muon_gated_ffn_grad(ctypes.byref(f), _ptr(x2), ldx, _ptr(dy2), ldy, _ptr(saved),
                                         saved.numel(), ctypes.byref(g), _ptr(ws), nbytes,
                                         _raw_stream(dev.index)))
    return (dx, *out)


# ------------------------------------------------------------------ autograd

class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.dtype, ctx.scale = weight.shape[0], weight.dtype, scale
        return muon_embedding(ids, weight, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        return None, muon_embedding_grad(dy, ids, ctx.vocab, ctx.scale, dtype=ctx.dtype), None


class _RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, rstd = muon_rms_norm(x, weight, residual, eps)
        ctx.save_for_backward(s, weight, rstd)
        ctx.set_materialize_grads(False)
        ctx.two = residual is not None
        return (y, s) if ctx.two else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        s, weight, rstd = ctx.saved_tensors
        if dy is None:
            return dsum, None, dsum, None
        dx, dw = muon_rms_norm_grad(dy, s, weight, rstd, dsum=dsum,
                                    want_dweight=ctx.needs_input_grad[1])
        return dx, dw, dx if ctx.two else None, None


class _GatedFFNFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, save=True):
        if not save:  # no backward pass will come
            return muon_gated_ffn(x, w_gate, w_up, w_down, activation)
        y, saved = muon_gated_ffn(x, w_gate, w_up, w_down, activation, save=True)
        ctx.save_for_backward(x, w_gate, w_up, w_down, saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = muon_gated_ffn_grad(dy, x, w_gate, w_up, w_down, saved, want_dx=need[0],
                                    want_dweights=any(need[1:4]))
        return (*grads, None, None)


class Embedding(torch.nn.Module):
    """Token embedding: scale · weight[ids], zero rows for ids outside
    [0, num_embeddings); the weight's gradient is dense and summed in a fixed
    order."""

    def __init__(self, num_embeddings: int, dim: int, scale: float = 1.0, device=None, dtype=None):
        super().__init__()
        self.scale = float(scale)
        self.weight = torch.nn.Parameter(torch.empty((num_embeddings, dim), device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, ids):
        return _EmbeddingFn.apply(ids, self.weight, self.scale)


class RMSNorm(torch.nn.Module):
    """RMS norm over the last dimension.  forward(x) returns the normed x;
    forward(x, residual) returns (normed x + residual, x + residual)."""

    def __init__(self, dim: int, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.eps = float(eps)
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        return _RMSNormFn.apply(x, self.weight, residual, self.eps)


class GatedFFN(torch.nn.Module):
    """Gated feed-forward block; its three matrices are Muon parameters."""

    def __init__(self, model: int, hidden: int, activation: str = "silu", device=None, dtype=None):
        super().__init__()
        if activation not in ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}; use one of {sorted(ACTIVATIONS)}")
        self.activation = activation
        kw = {"device": device, "dtype": dtype}
        self.w_gate = torch.nn.Parameter(torch.empty((hidden, model), **kw))
        self.w_up = torch.nn.Parameter(torch.empty((hidden, model), **kw))
        self.w_down = torch.nn.Parameter(torch.empty((model, hidden), **kw))
        for w in (self.w_gate, self.w_up, self.w_down):
            torch.nn.init.normal_(w, std=1.0 / math.sqrt(w.shape[1]))

    def forward(self, x):
        w = (self.w_gate, self.w_up, self.w_down)
        # always through the autograd function: it refuses forward-mode tangents,
        # which the plain call would drop
        return _GatedFFNFn.apply(x, *w, self.activation,
                                 torch.is_grad_enabled() and any(t.requires_grad for t in (x, *w)))
