"""Refusals and sizes of the layer entry points (no GPU needed): every check
runs on the host before any HIP call, so invalid calls are made with made-up
addresses and must return before anything is enqueued."""
import ctypes

import pytest
import torch

import muon_newton_schulz_06_amd as mns
from muon_newton_schulz_06_amd import layers

INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 1, 2, 3, 4
A, B, C, D, S, W, Y, Z = (0x10000000 * k for k in range(1, 9))
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    return layers._lib()


def embed(L, **kw):
    a = dict(ids=A, nb=8, tokens=4, weight=B, ldw=16, vocab=10, dim=16, scale=1.0, out=C, ldo=16, dt=F32)
    a.update(kw)
    return L.muon_embedding(a["ids"], a["nb"], a["tokens"], a["weight"], a["ldw"], a["vocab"], a["dim"],
                            a["scale"], a["out"], a["ldo"], a["dt"], None)


def embed_grad(L, **kw):
    a = dict(dy=A, ldy=16, ids=B, nb=8, tokens=4, vocab=10, dim=16, scale=1.0, dw=C, ldw=16, dt=F32, wdt=F32,
             acc=0, ws=W, n=1 << 20)
    a.update(kw)
    return L.muon_embedding_grad(a["dy"], a["ldy"], a["ids"], a["nb"], a["tokens"], a["vocab"], a["dim"],
                                 a["scale"], a["dw"], a["ldw"], a["dt"], a["wdt"], a["acc"], a["ws"], a["n"], None)


def norm(L, **kw):
    a = dict(x=A, ldx=16, r=B, ldr=16, w=C, wdt=F32, eps=1e-6, y=D, ldy=16, s=S, lds=16, rstd=W, tokens=4,
             dim=16, dt=F32)
    a.update(kw)
    return L.muon_rms_norm(a["x"], a["ldx"], a["r"], a["ldr"], a["w"], a["wdt"], a["eps"], a["y"], a["ldy"],
                           a["s"], a["lds"], a["rstd"], a["tokens"], a["dim"], a["dt"], None)


def norm_grad(L, **kw):
    a = dict(dy=A, ldy=16, s=B, lds=16, w=C, wdt=F32, rstd=D, ds=None, ldd=0, dx=S, ldx=16, dw=Y, acc=0, tokens=4,
             dim=16, dt=F32, ws=W, n=1 << 20)
    a.update(kw)
    return L.muon_rms_norm_grad(a["dy"], a["ldy"], a["s"], a["lds"], a["w"], a["wdt"], a["rstd"], a["ds"],
                                a["ldd"], a["dx"], a["ldx"], a["dw"], a["acc"], a["tokens"], a["dim"], a["dt"],
                                a["ws"], a["n"], None)


def ffn(L, grad=False, **kw):
    a = dict(tokens=4, model=16, hidden=32, wg=A, wu=B, wd=C, ldg=16, ldu=16, ldd=32, dt=BF16, act=0, x=D, ldx=16,
             y=S, ldy=16, saved=W, ns=1 << 20, ws=Y, n=1 << 20, dx=S, dwg=Z, dwu=Z + 0x100000, dwd=Z + 0x200000,
             gdt=BF16, acc=0, dy=S + 0x8000000, lddx=16)
    a.update(kw)
    f = layers.MuonFfn(a["tokens"], a["model"], a["hidden"], a["wg"], a["wu"], a["wd"], a["ldg"], a["ldu"], a["ldd"],
                       a["dt"], a["act"])
    if not grad:
        return L.muon_gated_ffn(ctypes.byref(f), a["x"], a["ldx"], a["y"], a["ldy"], a["saved"], a["ns"], a["ws"],
                                a["n"], None)
    g = layers.MuonFfnGrads(a["dx"], a["dwg"], a["dwu"], a["dwd"], a["lddx"], 16, 16, 32, a["gdt"], a["acc"])
    return L.muon_gated_ffn_grad(ctypes.byref(f), a["x"], a["ldx"], a["dy"], a["ldy"], a["saved"], a["ns"],
                                 ctypes.byref(g), a["ws"], a["n"], None)


COMMON = [(dict(tokens=-1), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED), (dict(dt=7), INVALID)]
CALLS = {
    embed: COMMON + [
        (dict(nb=2), INVALID), (dict(vocab=0), INVALID), (dict(dim=0), INVALID), (dict(scale=float("nan")), INVALID),
        (dict(ids=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(ldw=15), INVALID),
        (dict(ldo=15), INVALID), (dict(weight=B + 2), INVALID), (dict(ids=A + 4), INVALID), (dict(out=B + 64), ALIAS),
        (dict(out=A), ALIAS), (dict(dim=(1 << 20) + 1, ldw=1 << 21, ldo=1 << 21), UNSUPPORTED),
        (dict(vocab=(1 << 24) + 1), UNSUPPORTED), (dict(ldw=(1 << 32) + 1), UNSUPPORTED)],
    embed_grad: COMMON + [
        (dict(wdt=9), INVALID), (dict(dw=None), INVALID), (dict(dy=None), INVALID), (dict(ldw=3), INVALID),
        (dict(ws=None), WORKSPACE), (dict(ws=W + 8), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=A), ALIAS),
        (dict(dw=A), ALIAS), (dict(scale=float("inf")), INVALID)],
    norm: COMMON + [
        (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(r=None), INVALID), (dict(w=None), INVALID),
        (dict(y=S), ALIAS), (dict(y=A + 64), ALIAS), (dict(y=A, ldy=17), ALIAS), (dict(rstd=A), ALIAS),
        (dict(w=D), ALIAS), (dict(x=None), INVALID), (dict(dim=0), INVALID), (dict(wdt=5), INVALID)],
    norm_grad: COMMON + [
        (dict(dx=B), ALIAS), (dict(dx=A + 4), ALIAS), (dict(ws=None), WORKSPACE), (dict(n=32), WORKSPACE),
        (dict(rstd=None), INVALID), (dict(s=None), INVALID), (dict(dw=C), ALIAS), (dict(ldx=8), INVALID)],
    ffn: COMMON + [
        (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(model=0), INVALID), (dict(hidden=0), INVALID),
        (dict(wg=None), INVALID), (dict(ldd=31), INVALID), (dict(x=D + 1), INVALID), (dict(y=D), ALIAS),
        (dict(y=A), ALIAS), (dict(saved=W + 16), WORKSPACE), (dict(ns=64), WORKSPACE), (dict(n=0), WORKSPACE),
        (dict(ws=W), ALIAS), (dict(ws=None), WORKSPACE), (dict(hidden=(1 << 20) + 1, ldd=1 << 21), UNSUPPORTED)],
}


@pytest.mark.parametrize("call,kw,status", [(c, k, s) for c, ks in CALLS.items() for k, s in ks])
def test_refusals(L, call, kw, status):
    assert call(L, **kw) == status
    assert L.muon_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(saved=None), WORKSPACE), (dict(ns=64), WORKSPACE), (dict(n=0), WORKSPACE), (dict(dwu=None), INVALID),
    (dict(gdt=4), INVALID), (dict(dx=D), ALIAS), (dict(dwg=A), ALIAS), (dict(dwu=Z), ALIAS), (dict(dy=None), INVALID),
    (dict(lddx=8), INVALID), (dict(ws=W), ALIAS)])
def test_ffn_grad_refusals(L, kw, status):
    assert ffn(L, grad=True, **kw) == status
    assert L.muon_last_error().decode()


def test_nothing_to_do_needs_no_device(L):
    """Calls without work return before any HIP call, whatever the pointers."""
    assert embed(L, tokens=0, ids=None, weight=None, out=None) == 0
    assert embed_grad(L, tokens=0, ids=None, dy=None, acc=1, ws=None, n=0) == 0
    assert norm(L, tokens=0, x=None, r=None, y=None, s=None) == 0
    assert ffn(L, tokens=0, x=None, y=None, saved=None, ws=None) == 0
    assert ffn(L, grad=True, tokens=0, acc=1, x=None, dy=None, saved=None, ws=None, dx=None) == 0


def test_header_and_exports(L):
    """Every function the header declares is exported, and takes as many
    arguments as the binding gives it."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "muon_layers.h"), encoding="utf-8") as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    found = re.findall(r"muon_status_t\s+(muon_\w+)\s*\(([^)]*)\)", text)
    assert len(found) == 10
    for name, args in found:
        assert len(getattr(L, name).argtypes) == args.count(",") + 1, name


def test_sizes():
    n = mns.gated_ffn_saved_size(100, 64, 33)
    assert n >= 100 * 40 * 2 * 3 and n % 256 == 0
    assert mns.gated_ffn_saved_size(100, 64, 33, torch.float32) >= 100 * 40 * 4 * 3
    assert mns.gated_ffn_workspace_size(100, 64, 33) >= 100 * 40 * 2
    assert mns.gated_ffn_workspace_size(100, 64, 33, grad=True) >= 2 * 100 * 40 * 2
    assert mns.gated_ffn_saved_size(0, 64, 33) == 0
    with pytest.raises(TypeError):
        mns.gated_ffn_saved_size(1, 8, 8, torch.float16)
    with pytest.raises(mns.MuonError):
        mns.gated_ffn_workspace_size(1, 0, 8)


def test_binding_refuses_cpu_tensors_and_bad_arguments():
    x, w = torch.zeros((2, 8)), torch.zeros((4, 8))
    with pytest.raises(ValueError, match="CUDA/HIP"):
        mns.muon_embedding(torch.zeros(2, dtype=torch.int64), w)
    with pytest.raises(ValueError, match="CUDA/HIP"):
        mns.muon_embedding_grad(x, torch.zeros(2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="CUDA/HIP"):
        mns.muon_rms_norm(x, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA/HIP"):
        mns.muon_rms_norm_grad(x, x, torch.ones(8), torch.ones(2))
    with pytest.raises(ValueError, match="CUDA/HIP"):
        mns.muon_gated_ffn(x, w, w, w.t())
    with pytest.raises(ValueError, match="activation"):
        mns.GatedFFN(8, 16, "relu")
