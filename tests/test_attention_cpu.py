"""Refusals, sizes and bindings of the attention entry points, and their fp64
oracle (no GPU needed): every check runs on the host before any HIP call, so
invalid calls are made with made-up addresses and must return before anything
is enqueued."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwad

import muon_newton_schulz_06_amd as mns
import oracle.attention as oa
from muon_newton_schulz_06_amd import attention

INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 1, 2, 3, 4
A, B, C, D, S, W, Y, Z = (0x100000000 * k for k in range(1, 9))
F32, BF16 = 0, 1
I3 = attention._i64x3


@pytest.fixture(scope="module")
def L():
    return attention._lib()


def rotary(L, **kw):
    a = dict(batch=2, tokens=4, dim=64, rot=64, freqs=C, pos=D, ps=4, start=0, nb=8, inter=0, scale=1.0, dt=BF16, q=A,
             qo=B, heads=4, qs=(1024, 256, 64), qos=(1024, 256, 64), k=S, ko=W, kh=2, ks=(512, 128, 64),
             kos=(512, 128, 64), n=2, r=True, t=True)
    a.update(kw)
    r = attention.MuonRotary(a["batch"], a["tokens"], a["dim"], a["rot"], a["freqs"], a["pos"], a["ps"], a["start"],
                             a["nb"], a["inter"], a["scale"], a["dt"])
    t = (attention.MuonRotaryHeads * 2)(
        attention.MuonRotaryHeads(a["q"], a["qo"], a["heads"], I3(*a["qs"]), I3(*a["qos"])),
        attention.MuonRotaryHeads(a["k"], a["ko"], a["kh"], I3(*a["ks"]), I3(*a["kos"])))
    codes = {f(ctypes.byref(r) if a["r"] else None, t if a["t"] else None, a["n"], None)
             for f in (L.muon_rotary, L.muon_rotary_grad)}
    assert len(codes) == 1
    return codes.pop()


def dropout(L, **kw):
    a = dict(x=A, ldx=64, r=B, ldr=64, p=0.5, seed=1, off=2, offd=C, y=D, ldy=64, rows=4, cols=64, dt=BF16)
    a.update(kw)
    return L.muon_dropout(a["x"], a["ldx"], a["r"], a["ldr"], a["p"], a["seed"], a["off"], a["offd"], a["y"], a["ldy"],
                          a["rows"], a["cols"], a["dt"], None)


def dropout_grad(L, **kw):
    a = dict(x=A, ldx=64, p=0.5, seed=1, off=2, offd=C, y=D, ldy=64, rows=4, cols=64, dt=BF16)
    a.update(kw)
    return L.muon_dropout_grad(a["x"], a["ldx"], a["p"], a["seed"], a["off"], a["offd"], a["y"], a["ldy"], a["rows"],
                               a["cols"], a["dt"], None)


def diff(L, grad=False, **kw):
    a = dict(batch=2, queries=5, keys=7, heads=4, kv=2, dim=64, q=A, k=B, v=C, lam=D, offsets=None, seqs=0, scale=0.125,
             causal=1, dt=BF16, out=S, saved=W, ns=1 << 22, ws=Y, n=1 << 22, dout=Z, dq=A + (1 << 28), dk=B + (1 << 28),
             dv=C + (1 << 28), dlam=D + (1 << 28), f=True, g=True)
    a.update(kw)
    d, h, kv = a["dim"], a["heads"], a["kv"]
    st = lambda tokens, heads, dim: (tokens * heads * dim, heads * dim, dim)
    qs, ks, vs, os = (I3(*a.get(n, s)) for n, s in (
        ("qs", st(a["queries"], 2 * h, d)), ("ks", st(a["keys"], 2 * kv, d)), ("vs", st(a["keys"], kv, 2 * d)),
        ("os", st(a["queries"], h, 2 * d))))
    f = attention.MuonDiffAttention(a["batch"], a["queries"], a["keys"], h, kv, d, a["q"], a["k"], a["v"], a["lam"], qs,
                                    ks, vs, a["offsets"], a["seqs"], a["scale"], a["causal"], a["dt"])
    f = ctypes.byref(f) if a["f"] else None
    if not grad:
        return L.muon_diff_attention(f, a["out"], None if a.get("nostrides") else os, a["saved"], a["ns"], a["ws"], a["n"],
                                     None)
    g = attention.MuonDiffAttentionGrads(a["dq"], a["dk"], a["dv"], a["dlam"], I3(*a.get("dqs", qs)),
                                         I3(*a.get("dks", ks)), I3(*a.get("dvs", vs)))
    return L.muon_diff_attention_grad(f, a["dout"], None if a.get("nostrides") else os, a["out"], os, a["saved"], a["ns"],
                                      ctypes.byref(g) if a["g"] else None, a["ws"], a["n"], None)


BIG = 1 << 24
CALLS = {
    rotary: [
        (dict(r=False), INVALID), (dict(t=False), INVALID), (dict(n=0), INVALID), (dict(n=3), INVALID),
        (dict(batch=-1), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=BIG + 1), UNSUPPORTED),
        (dict(batch=BIG, tokens=2), UNSUPPORTED), (dict(dim=0), INVALID), (dict(dim=1025, rot=4), UNSUPPORTED),
        (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=66), INVALID), (dict(scale=math.nan), INVALID),
        (dict(scale=math.inf), INVALID), (dict(dt=2), INVALID), (dict(heads=-1), INVALID),
        (dict(heads=(1 << 16) + 1), UNSUPPORTED), (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
        (dict(q=A + 1), INVALID), (dict(qs=(1024, -256, 64)), INVALID), (dict(qs=((1 << 40) + 1, 256, 64)), UNSUPPORTED),
        (dict(qos=(1024, 0, 64)), ALIAS), (dict(qos=(1024, 256, 63)), ALIAS), (dict(freqs=None), INVALID),
        (dict(freqs=C + 4), INVALID), (dict(nb=2), INVALID), (dict(pos=D + 4), INVALID), (dict(ps=3), INVALID),
        (dict(qo=A + 64), ALIAS), (dict(qo=A, qos=(1024, 64, 256)), ALIAS), (dict(ko=A), ALIAS), (dict(qo=S), ALIAS),
        (dict(ko=B), ALIAS), (dict(qo=C), ALIAS), (dict(qo=D), ALIAS)],
    dropout: [
        (dict(rows=-1), INVALID), (dict(rows=BIG + 1), UNSUPPORTED), (dict(cols=0), INVALID),
        (dict(cols=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21, ldr=1 << 21), UNSUPPORTED), (dict(dt=5), INVALID),
        (dict(p=-0.1), INVALID), (dict(p=1.1), INVALID), (dict(p=math.nan), INVALID), (dict(x=None), INVALID),
        (dict(y=None), INVALID), (dict(ldx=63), INVALID), (dict(ldr=63), INVALID), (dict(ldy=63), INVALID),
        (dict(x=A + 1), INVALID), (dict(offd=C + 4), INVALID), (dict(y=A + 64), ALIAS), (dict(y=A, ldy=65), ALIAS),
        (dict(y=B, ldy=128), ALIAS), (dict(y=C), ALIAS)],
    dropout_grad: [
        (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dt=5), INVALID), (dict(p=2.0), INVALID),
        (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(ldy=1), INVALID), (dict(y=A + 2), ALIAS),
        (dict(y=C - 64), ALIAS)],
    diff: [
        (dict(f=False), INVALID), (dict(nostrides=True), INVALID), (dict(batch=-1), INVALID), (dict(queries=-1), INVALID),
        (dict(keys=-1), INVALID), (dict(keys=BIG + 1), UNSUPPORTED), (dict(heads=0), INVALID), (dict(kv=0), INVALID),
        (dict(kv=3), INVALID), (dict(heads=2, kv=4), INVALID), (dict(dim=0), INVALID), (dict(dim=129), UNSUPPORTED),
        (dict(dt=3), INVALID), (dict(batch=BIG, queries=2), UNSUPPORTED), (dict(batch=BIG, keys=2), UNSUPPORTED),
        (dict(heads=1 << 7, kv=1, queries=BIG), UNSUPPORTED), (dict(batch=1, heads=32, kv=32, queries=BIG), UNSUPPORTED),
        (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID),
        (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID), (dict(scale=1e-20), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
        (dict(v=None), INVALID), (dict(lam=None), INVALID), (dict(out=None), INVALID), (dict(q=A + 1), INVALID),
        (dict(lam=D + 2), INVALID), (dict(seqs=-1), INVALID), (dict(seqs=2, offsets=Z), INVALID),
        (dict(seqs=2, offsets=Z, batch=1), INVALID), (dict(seqs=2, offsets=None, batch=1, keys=5), INVALID),
        (dict(seqs=2, offsets=Z + 2, batch=1, keys=5), INVALID), (dict(ks=(1792, -256, 64)), INVALID),
        (dict(os=(2560, 0, 128)), ALIAS), (dict(os=(2560, 512, 127)), ALIAS), (dict(ws=None, q=A + 2), WORKSPACE),
        (dict(ws=Y + 8, q=A + 2), WORKSPACE), (dict(n=16, q=A + 2), WORKSPACE), (dict(ns=64), WORKSPACE),
        (dict(saved=W + 16), WORKSPACE), (dict(out=A), ALIAS), (dict(out=C), ALIAS), (dict(out=D), ALIAS),
        (dict(saved=A), ALIAS), (dict(ws=W, q=A + 2), ALIAS), (dict(ws=S, q=A + 2), ALIAS),
        (dict(batch=1 << 22, queries=1, heads=4, kv=4, keys=1, ns=1 << 50, n=1 << 50, q=A << 16, k=B << 16, v=C << 16,
              out=S << 16, saved=W << 16, ws=Y << 16), UNSUPPORTED)],
}


@pytest.mark.parametrize("call,kw,status", [(c, k, s) for c, ks in CALLS.items() for k, s in ks])
def test_refusals(L, call, kw, status):
    assert call(L, **kw) == status
    assert L.muon_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(g=False), INVALID), (dict(f=False), INVALID), (dict(nostrides=True), INVALID), (dict(dim=129), UNSUPPORTED),
    (dict(dout=None), INVALID), (dict(out=None), INVALID), (dict(dout=Z + 1), INVALID), (dict(saved=None), WORKSPACE),
    (dict(ns=64), WORKSPACE), (dict(n=64), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(dk=None), INVALID),
    (dict(dv=None), INVALID), (dict(dlam=D + (1 << 28) + 2), INVALID), (dict(dqs=(2560, 0, 64)), ALIAS),
    (dict(dks=(1792, 256, 32)), ALIAS), (dict(dq=A), ALIAS), (dict(dq=Z), ALIAS), (dict(dv=S), ALIAS),
    (dict(dk=A + (1 << 28)), ALIAS), (dict(dlam=D), ALIAS), (dict(dq=W), ALIAS), (dict(ws=Z), ALIAS),
    (dict(scale=0.0), INVALID), (dict(lam=None), INVALID)])
def test_diff_attention_grad_refusals(L, kw, status):
    assert diff(L, grad=True, **kw) == status
    assert L.muon_last_error().decode()


@pytest.mark.parametrize("kw,overlap", [
    # q and k of one projection in place: of several tokens, and of one token of several batch entries
    (dict(batch=2, tokens=4, q=A, qo=A, qs=(2048, 512, 64), qos=(2048, 512, 64), k=A + 512, ko=A + 512,
          ks=(2048, 512, 64), kos=(2048, 512, 64)), False),
    (dict(batch=3, tokens=1, q=A, qo=A, qs=(512, 512, 64), qos=(512, 512, 64), k=A + 512, ko=A + 512,
          ks=(512, 512, 64), kos=(512, 512, 64)), False),
    (dict(batch=3, tokens=1, q=A, qo=A, qs=(512, 7, 64), qos=(512, 7, 64), k=A + 510, ko=A + 510,
          ks=(512, 9, 64), kos=(512, 9, 64)), True),
    (dict(batch=3, tokens=1, q=A, qo=A, qs=(512, 7, 64), qos=(512, 7, 64), k=A + 512, ko=A + 512,
          ks=(500, 9, 64), kos=(500, 9, 64)), True)])
def test_interleaved_tensors(L, kw, overlap):
    """(heads 4 and 2 of 64 bf16; what is taken gets as far as the device)"""
    assert (rotary(L, **kw) == ALIAS) == overlap


def test_nothing_to_do_needs_no_device(L):
    """Calls without work return before any HIP call, whatever the pointers."""
    assert rotary(L, tokens=0, q=None, qo=None, k=None, ko=None, freqs=None, pos=None) == 0
    assert rotary(L, heads=0, kh=0, q=None, qo=None, k=None, ko=None, freqs=None, pos=None) == 0
    assert dropout(L, rows=0, x=None, r=None, y=None, offd=None) == 0
    assert dropout_grad(L, rows=0, x=None, y=None, offd=None) == 0
    assert diff(L, queries=0, q=None, out=None, lam=None) == 0
    assert diff(L, batch=0, q=None, k=None, v=None, out=None, lam=None) == 0
    assert diff(L, grad=True, dq=None, dk=None, dv=None, dlam=None) == 0
    assert diff(L, grad=True, batch=0, q=None, k=None, v=None, out=None, dout=None, lam=None, dlam=None, dq=None,
                dk=None, dv=None) == 0


def test_header_and_exports(L):
    """Every function the header declares is exported, and takes as many
    arguments as the binding gives it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "muon_attention.h"), encoding="utf-8") as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    found = re.findall(r"muon_status_t\s+(muon_\w+)\s*\(([^)]*)\)", text)
    assert len(found) == 8
    for name, args in found:
        assert len(getattr(L, name).argtypes) == args.count(",") + 1, name


def test_structs_match_the_header(tmp_path):
    """The binding's structures have the header's sizes and field offsets."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = {"muon_rotary_t": attention.MuonRotary, "muon_rotary_heads_t": attention.MuonRotaryHeads,
             "muon_diff_attention_t": attention.MuonDiffAttention,
             "muon_diff_attention_grads_t": attention.MuonDiffAttentionGrads}
    names = {"in_": "in", "lam": "lambda", "dlam": "dlambda"}
    lines = [f'printf("%zu ", sizeof({c}));' + "".join(
        f'printf("%zu ", offsetof({c}, {names.get(n, n)}));' for n, _ in t._fields_) for c, t in pairs.items()]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon_attention.h"\nint main(void) {'
                   + "\n".join(lines) + "return 0; }\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), "-o", tmp_path / "s", src],
                   check=True)
    got = [int(v) for v in subprocess.run([tmp_path / "s"], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for t in pairs.values():
        want += [ctypes.sizeof(t)] + [getattr(t, n).offset for n, _ in t._fields_]
    assert got == want


def test_sizes():
    n = mns.diff_attention_saved_size(2, 100, 100, 6, 2, 33)
    assert n >= 2 * 6 * 100 * (2 * 4 + 72 * 2) and n % 256 == 0
    assert mns.diff_attention_saved_size(2, 100, 100, 6, 2, 33, torch.float32) >= 2 * 6 * 100 * (2 * 4 + 68 * 4)
    assert mns.diff_attention_saved_size(0, 100, 100, 6, 2, 33) == 0
    assert mns.diff_attention_workspace_size(1, 1, 0, 2, 2, 64) >= 0
    # room for aligned copies of q, k, v (and dout), one more list for a packed batch
    one = mns.diff_attention_workspace_size(1, 700, 700, 6, 2, 33)
    assert one >= 700 * (12 + 4 + 4) * 40 * 2
    assert mns.diff_attention_workspace_size(1, 700, 700, 6, 2, 33, sequences=5) > one - (64 << 20)
    assert mns.diff_attention_workspace_size(1, 700, 700, 6, 2, 33, grad=True) >= one + 700 * 6 * 72 * 2 - (64 << 20)
    with pytest.raises(TypeError):
        mns.diff_attention_saved_size(2, 100, 100, 6, 2, 33, torch.float16)
    with pytest.raises(mns.MuonError):
        mns.diff_attention_workspace_size(2, 100, 100, 6, 4, 33)


# ------------------------------------------------------------------ binding

def test_binding_refuses():
    q, k, v, lam = torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 2, 16), torch.zeros(2)
    for call in (lambda: mns.muon_rotary(q, k, torch.zeros(4, dtype=torch.float64)),
                 lambda: mns.muon_rotary_grad(q, k, torch.zeros(4, dtype=torch.float64)),
                 lambda: mns.muon_dropout(q, 0.5, 1), lambda: mns.muon_dropout_grad(q, 0.5, 1),
                 lambda: mns.muon_diff_attention(q, k, v, lam),
                 lambda: mns.muon_diff_attention_grad(q, q, k, v, lam, q, torch.zeros(1, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="CUDA/HIP device"):
            call()


@pytest.fixture
def free(monkeypatch):
    """Argument checks behind the device's: CPU tensors pass, the library's
    calls are noted and do nothing."""
    calls = []

    class Fake:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real_lib, name)

            def call(*a):
                calls.append((name, a))
                return 0
            return call
    real_lib = attention._lib()
    fake = Fake()
    monkeypatch.setattr(attention, "_lib", lambda: fake)
    monkeypatch.setattr(attention, "_device", lambda t, name: t.device)
    from muon_newton_schulz_06_amd import layers
    monkeypatch.setattr(attention, "_on", lambda dev, stream: layers._HERE)
    monkeypatch.setattr(attention, "_raw_stream", lambda i: 0)
    import contextlib
    monkeypatch.setattr(attention, "_workspace", lambda n, dev, user, stream: contextlib.nullcontext((None, n)))
    return calls


FR = torch.zeros(4, dtype=torch.float64)
X = torch.zeros(2, 3, 4, 8)


@pytest.mark.parametrize("kw,error", [
    (dict(q=X.half()), TypeError), (dict(q=X[0, 0]), ValueError), (dict(k=X.bfloat16()), TypeError),
    (dict(freqs=FR.float()), TypeError), (dict(freqs=FR[None]), ValueError), (dict(freqs=torch.zeros(8).double()[::2]), ValueError),
    (dict(positions=torch.zeros(3)), TypeError), (dict(positions=torch.zeros(4, dtype=torch.int64)), ValueError),
    (dict(positions=torch.zeros(3, 3, dtype=torch.int64)), ValueError), (dict(k=X[:1]), ValueError),
    (dict(k=X[:, :2]), ValueError), (dict(k=X[..., :4]), ValueError), (dict(k=X[0]), ValueError),
    (dict(q_out=X[..., :4]), ValueError), (dict(q_out=X.bfloat16()), TypeError),
    (dict(q_out=torch.zeros(2, 3, 8, 4).transpose(2, 3)), ValueError)])
def test_rotary_arguments(free, kw, error):
    a = dict(q=X, k=X.clone(), freqs=FR)
    with pytest.raises(error):
        mns.muon_rotary(**{**a, **kw})
    assert not free
    mns.muon_rotary(**a)
    assert [n for n, _ in free] == ["muon_rotary"]


@pytest.mark.parametrize("positions,stride,nb", [
    (torch.arange(3), 0, 8), (torch.arange(3)[None], 0, 8), (torch.arange(3)[None].expand(2, 3), 0, 8),
    (torch.arange(6).reshape(2, 3), 3, 8), (torch.arange(6, dtype=torch.int32).reshape(3, 2).t(), 3, 4),
    (torch.arange(20).reshape(2, 10)[:, 2:5], 10, 8), (None, 0, 0)])
def test_rotary_positions(free, positions, stride, nb):
    mns.muon_rotary(X, None, FR, positions=positions, start=5)
    (name, (r, arr, n, _)), = free
    r = r._obj
    assert n == 1 and r.position_stride == stride and r.position_bytes == nb and r.start == 5
    assert bool(r.positions) == (positions is not None)


T = dict(q=torch.zeros(2, 3, 8, 6), k=torch.zeros(2, 5, 4, 6), v=torch.zeros(2, 5, 2, 12), lam=torch.zeros(4))


@pytest.mark.parametrize("kw,error", [
    (dict(q=T["q"].half()), TypeError), (dict(k=T["k"].bfloat16()), TypeError), (dict(lam=T["lam"].double()), TypeError),
    (dict(q=T["q"][0]), ValueError), (dict(q=T["q"][:, :, :7]), ValueError), (dict(k=T["k"][:1]), ValueError),
    (dict(k=T["k"][..., :5]), ValueError), (dict(v=T["v"][..., :6]), ValueError), (dict(v=T["v"][:, :4]), ValueError),
    (dict(lam=torch.zeros(8)), ValueError), (dict(lam=torch.zeros(())), ValueError),
    (dict(offsets=torch.zeros(2, dtype=torch.int32)), ValueError), (dict(out=torch.zeros(2, 3, 4, 6)), ValueError),
    (dict(out=torch.zeros(2, 3, 4, 12).bfloat16()), TypeError)])
def test_attention_arguments(free, kw, error):
    with pytest.raises(error):
        mns.muon_diff_attention(**{**T, **kw})
    assert not free
    mns.muon_diff_attention(**T)
    (name, (f, *_)), = free
    f = f._obj
    assert name == "muon_diff_attention" and (f.batch, f.queries, f.keys, f.heads, f.kv_heads, f.dim) == (2, 3, 5, 4, 2, 6)
    assert f.scale == pytest.approx(6 ** -0.5) and f.causal == 1 and f.sequences == 0


@pytest.mark.parametrize("offsets,error", [
    (torch.zeros(2), TypeError), (torch.zeros(2, dtype=torch.int64), TypeError),
    (torch.zeros(1, dtype=torch.int32), ValueError), (torch.zeros(2, 2, dtype=torch.int32), ValueError)])
def test_attention_offsets(free, offsets, error):
    one = dict(q=T["q"][0], k=T["k"][0, :3], v=T["v"][0, :3], lam=T["lam"])
    with pytest.raises(error):
        mns.muon_diff_attention(**one, offsets=offsets)
    mns.muon_diff_attention(**one, offsets=torch.zeros(6, dtype=torch.int32)[::2])
    (name, (f, *_)), = free
    assert f._obj.sequences == 2


@pytest.mark.parametrize("kw,error", [
    (dict(dout=torch.zeros(2, 3, 4, 6)), ValueError), (dict(out=torch.zeros(2, 3, 2, 12)), ValueError),
    (dict(dout=torch.zeros(2, 3, 4, 12).bfloat16()), TypeError), (dict(saved=torch.zeros(64)), TypeError),
    (dict(saved=torch.zeros(64, dtype=torch.uint8)[::2]), ValueError)])
def test_attention_grad_arguments(free, kw, error):
    o = torch.zeros(2, 3, 4, 12)
    a = dict(dout=o, **T, out=o, saved=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(error):
        mns.muon_diff_attention_grad(**{**a, **kw})
    assert not free
    dq, dk, dv, dlam = mns.muon_diff_attention_grad(**a, want_dq=False)
    assert dq is None and dk.shape == T["k"].shape and dv.shape == T["v"].shape and dlam.shape == (4,)
    (name, args), = free
    g = args[7]._obj
    assert not g.dq and g.dk and g.dv and g.dlam


@pytest.mark.parametrize("kw,error", [
    (dict(x=X.half()), TypeError), (dict(residual=X[0]), ValueError), (dict(residual=X.bfloat16()), TypeError),
    (dict(offset=torch.zeros(1)), TypeError), (dict(offset=torch.zeros(2, dtype=torch.int64)), ValueError),
    (dict(out=X[0]), ValueError), (dict(x=torch.zeros(())), ValueError)])
def test_dropout_arguments(free, kw, error):
    with pytest.raises(error):
        mns.muon_dropout(**{**dict(x=X, p=0.5, seed=1), **kw})
    assert not free
    mns.muon_dropout(X, 0.5, -1, offset=-2)
    assert free[0][1][5] == 2 ** 64 - 1 and free[0][1][6] == 2 ** 64 - 2  # taken modulo 2^64


# ------------------------------------------------------------------ modules

def test_rotary_frequencies():
    f, s = mns.rotary_frequencies(8, 100.0)
    assert s == 1.0 and f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75],
                                                                                   dtype=torch.float64), rtol=1e-15)
    g, s = mns.rotary_frequencies(8, 100.0, "linear", factor=4.0)
    assert s == 1.0 and torch.equal(g, f / 4)
    g, s = mns.rotary_frequencies(8, 100.0, "base", factor=4.0)
    assert s == 1.0 and g[0] == 1 and g[-1] == pytest.approx(float(f[-1]) / 4, rel=1e-12)
    assert torch.all(g[1:] < f[1:]) and torch.all(g[1:-1] > f[1:-1] / 4)
    f, _ = mns.rotary_frequencies(128)
    g, s = mns.rotary_frequencies(128, scaling="yarn", factor=16.0, original_length=4096)
    assert s == pytest.approx(0.1 * math.log(16) + 1)
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.9], f[turns < 0.9] / 16, rtol=1e-15)
    assert torch.all(g <= f) and torch.all(g >= f / 16)
    assert mns.rotary_frequencies(128, scaling="yarn", factor=1.0, original_length=4096)[1] == 1.0
    for kw in (dict(dim=7), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, factor=0.0), dict(dim=8, scaling="other"),
               dict(dim=2, scaling="base"), dict(dim=8, scaling="yarn")):
        with pytest.raises(ValueError):
            mns.rotary_frequencies(**kw)


def test_modules_refuse():
    with pytest.raises(ValueError):
        mns.Rotary(8, rotated=10)
    with pytest.raises(ValueError):
        mns.Rotary(8)(torch.zeros(1, 2, 2, 6))
    with pytest.raises(ValueError):
        mns.Dropout(1.5)
    with pytest.raises(ValueError):
        mns.DiffAttention(4, 8, kv_heads=3)
    with pytest.raises(ValueError):
        mns.DiffAttention(2, 8)(torch.zeros(1, 2, 4, 6), torch.zeros(1, 2, 4, 8), torch.zeros(1, 2, 2, 16))


def test_dropout_module_without_dropping():
    x, r = torch.randn(3, 4), torch.randn(3, 4)
    for m in (mns.Dropout(0.0), mns.Dropout(0.7).eval()):
        assert m(x) is x and torch.equal(m(x, r), x + r) and int(m.calls) == 0


def test_dropout_module_seeds():
    """Drawn apart, repeatable by torch's seed, restored with the state."""
    torch.manual_seed(5)
    a, b = mns.Dropout(0.5), mns.Dropout(0.5)
    torch.manual_seed(5)
    assert a.seed != b.seed and mns.Dropout(0.5).seed == a.seed and mns.Dropout(0.5, seed=9).seed == 9
    a.calls += 7
    b.load_state_dict(a.state_dict())
    assert b.seed == a.seed and int(b.calls) == 7


def test_rotary_frequencies_outlive_inference_mode(free):
    """Copies made where no gradients are recorded serve a training pass later."""
    with torch.inference_mode():
        rot = mns.Rotary(8)
        rot(X.clone())
    q = X.clone().requires_grad_()
    rot(q)
    assert not rot.freqs.is_inference() and not any(f.is_inference() for f in rot._here.values())


def test_lambda():
    m = mns.DiffAttention(3, 8, lambda_init=0.3)
    lam = m.lam()
    want = math.exp(float(m.lambda_q1 @ m.lambda_k1)) - math.exp(float(m.lambda_q2 @ m.lambda_k2)) + 0.3
    assert lam.shape == (3,) and lam.dtype == torch.float32 and torch.allclose(lam, torch.full((3,), want), rtol=1e-5)
    lam.sum().backward()
    assert torch.allclose(m.lambda_q1.grad, 3 * math.exp(float(m.lambda_q1 @ m.lambda_k1)) * m.lambda_k1.detach(), rtol=1e-5)


def test_saved_only_where_a_backward_pass_comes(free):
    for grads in (False, True):
        q = T["q"].clone().requires_grad_(grads)
        y = attention._DiffAttentionFn.apply(q, T["k"], T["v"], T["lam"], True, None, None, grads)
        assert y.requires_grad == grads
        assert bool(free[-1][1][3]) == grads


def test_tangents_are_refused(free):
    """Forward-mode derivatives are not defined, and never answered with zero."""
    with fwad.dual_level():
        d = lambda t: fwad.make_dual(t, torch.ones_like(t))
        for call in (lambda: mns.Rotary(8)(d(X), X), lambda: mns.Dropout(0.5)(d(X)),
                     lambda: attention._DiffAttentionFn.apply(d(T["q"]), T["k"], T["v"], T["lam"], True, None, None, False)):
            with pytest.raises(NotImplementedError):
                call()


# ------------------------------------------------------------------- oracle

def test_philox_known_answers():
    """Three answers published with the generator's definition."""
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in oa.philox4x32_10(np.array([counter]), key)[0]) == want


def test_oracle_rotary():
    r = np.random.RandomState(0)
    x, f, pos = r.randn(2, 5, 3, 10), np.array([1.0, 0.3, 0.01]), r.randint(-50, 1 << 20, (2, 5))
    for inter in (False, True):
        y = oa.rotary(x, f, pos, inter)
        assert np.allclose(oa.rotary(y, f, pos, inter, inverse=True), x, atol=1e-12)
        z = x[..., 0:6:2] + 1j * x[..., 1:6:2] if inter else x[..., :3] + 1j * x[..., 3:6]
        w = z * np.exp(1j * pos[:, :, None, None] * f)
        got = y[..., 0:6:2] + 1j * y[..., 1:6:2] if inter else y[..., :3] + 1j * y[..., 3:6]
        assert np.allclose(got, w, atol=1e-12) and np.array_equal(y[..., 6:], x[..., 6:])


def test_oracle_attention():
    """Against torch's autograd in fp64, and against central differences."""
    r = np.random.RandomState(1)
    q, k, v, lam, do = r.randn(1, 6, 8, 4), r.randn(1, 9, 4, 4), r.randn(1, 9, 2, 8), r.rand(4), r.randn(1, 6, 4, 8)

    def f(q, k, v, lam, causal):
        k, v = k.repeat_interleave(2, 2), v.repeat_interleave(2, 2)  # (maps of a group's heads, below)
        out = []
        for h in range(4):
            g = h // 2
            m = [torch.einsum("btd,bsd->bts", q[:, :, 2 * h + i], k[:, :, 2 * (2 * g + i)]) / 2 for i in (0, 1)]
            if causal:
                m = [s.masked_fill(torch.ones(6, 9).triu(4).bool(), -math.inf) for s in m]
            p = [s.softmax(-1) for s in m]
            out.append(torch.einsum("bts,bsd->btd", p[0] - lam[h] * p[1], v[:, :, h]))
        return torch.stack(out, 2)
    for causal in (False, True):
        ts = [torch.tensor(a, requires_grad=True) for a in (q, k, v, lam)]
        y = f(*ts, causal)
        got, bound = oa.diff_attention(q, k, v, lam, causal)
        assert np.allclose(got, y.detach().numpy(), atol=1e-12) and np.all(bound < 1e-3)
        y.backward(torch.tensor(do))
        grads, err = oa.diff_attention_grad(do, q, k, v, lam, causal)
        for n, t in zip(("dq", "dk", "dv", "dlam"), ts):
            assert np.allclose(grads[n], t.grad.numpy(), atol=1e-12), n
            assert np.all(err[n] < 1e-2), n


def test_oracle_packed():
    r = np.random.RandomState(2)
    q, k, v, lam = r.randn(1, 20, 4, 4), r.randn(1, 20, 2, 4), r.randn(1, 20, 1, 8), r.rand(2)
    assert oa.spans(20, [-3, 4, 4, 2, 30, 17]) == [(0, 4), (4, 4), (4, 4), (4, 20), (20, 20)]
    out, _ = oa.diff_attention(q, k, v, lam, offsets=[2, 7, 7, 19])
    assert not out[:, :2].any() and not out[:, 19:].any()
    for a, b in ((2, 7), (7, 19)):
        one, _ = oa.diff_attention(q[:, a:b], k[:, a:b], v[:, a:b], lam)
        assert np.array_equal(out[:, a:b], one)
