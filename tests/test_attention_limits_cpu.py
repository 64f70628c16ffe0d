"""Launch sizes of the attention entry points at their documented limits (no
GPU needed): a stand-in for the runtime's launch, loaded ahead of it into a
child process, notes each launch and starts nothing."""
import json
import os
import subprocess
import sys

import pytest
from test_launch_limits_cpu import STANDIN, check

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from muon_newton_schulz_06_amd import attention as at
L = at._lib()
P = [k << 50 for k in range(1, 16)]
I3, B, vp = at._i64x3, ctypes.byref, ctypes.c_void_p
def dense(tokens, heads, dim):
    return I3(tokens * heads * dim, heads * dim, dim)
def rotary(batch, tokens, heads, kv, dim, rot, inter, dt):
    r = at.MuonRotary(batch, tokens, dim, rot, P[0], P[1], tokens, 0, 8, inter, 1.0, dt)
    t = (at.MuonRotaryHeads * 2)(at.MuonRotaryHeads(P[2], P[3], heads, dense(tokens, heads, dim), dense(tokens, heads, dim)),
                                 at.MuonRotaryHeads(P[4], P[5], kv, dense(tokens, kv, dim), dense(tokens, kv, dim)))
    return L.muon_rotary(B(r), t, 2, None) or L.muon_rotary_grad(B(r), t, 2, None)
def dropout(rows, cols, pad, res, dt):
    return (L.muon_dropout(P[0], cols + pad, P[1] if res else None, cols + pad, 0.5, 1, 2, P[2], P[3], cols + pad, rows, cols,
                           dt, None)
            or L.muon_dropout_grad(P[0], cols + pad, 0.5, 1, 2, P[2], P[3], cols + pad, rows, cols, dt, None))
def attention(batch, queries, keys, heads, kv, dim, seqs, causal, dt):
    qs, ks, vs, os = (dense(queries, 2 * heads, dim), dense(keys, 2 * kv, dim), dense(keys, kv, 2 * dim),
                      dense(queries, heads, 2 * dim))
    f = at.MuonDiffAttention(batch, queries, keys, heads, kv, dim, P[0], P[1], P[2], P[3], qs, ks, vs, P[4] if seqs else None,
                             seqs, 0.125, causal, dt)
    n = ctypes.c_size_t(0)
    for dout in (None, P[10]):
        assert L.muon_diff_attention_workspace_size(B(f), dout, os, B(n)) == 0
        print("bytes", n.value, flush=True)
    s = L.muon_diff_attention(B(f), P[5], os, P[6], 1 << 48, P[7], 1 << 48, None)
    g = at.MuonDiffAttentionGrads(P[11], P[12], P[13], P[14], qs, ks, vs)
    return s or L.muon_diff_attention_grad(B(f), P[10], os, P[5], os, P[6], 1 << 48, B(g), P[7], 1 << 48, None)
for name, *args in json.loads(sys.argv[3]):
    print("call", json.dumps([name, *args]), flush=True)
    print("status", globals()[name](*args), flush=True)
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """{call: ([(grid, block), ..], [workspace bytes of both passes])}"""
    tmp = tmp_path_factory.mktemp("standin")
    src, so = tmp / "standin.c", tmp / "standin.so"
    src.write_text(STANDIN)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, src], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-c", CHILD, so, ROOT, json.dumps(calls)], capture_output=True, text=True,
                           timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        out, call = {}, None
        for line in r.stdout.splitlines():
            word, *rest = line.split(" ", 1)
            if word == "call":
                call = rest[0]
                out[call] = ([], [])
            elif word == "status":
                assert rest == ["0"], (call, line)
            elif word == "bytes":
                out[call][1].append(int(rest[0]))
            else:
                n = [int(v) for v in line.split()]
                out[call][0].append((n[:3], n[3:]))
        return out
    return run


def test_rotary(launches):
    calls = [["rotary", b, t, h, kv, dim, rot, inter, dt] for b, t in ((1, 1), (1, 1 << 24), (1 << 24, 1), (4096, 4096))
             for h, kv in ((1, 1), (64, 8), (1 << 16, 1)) for dim, rot in ((2, 2), (64, 64), (128, 2), (1024, 1024))
             for inter in (0, 1) for dt in (0, 1) if b * t * h * dim * 2 < 1 << 44]
    check({c: ls for c, (ls, _) in launches(calls).items()}, least=2)


def test_dropout(launches):
    calls = [["dropout", r, c, pad, res, dt] for r in (1, 7, 1 << 16, (1 << 16) + 1, 1 << 24)
             for c in (1, 3, 4, 1000, 1 << 14, 1 << 20) for pad in (0, 1) for res in (0, 1) for dt in (0, 1)
             if r * (c + 1) < 1 << 38]
    check({c: ls for c, (ls, _) in launches(calls).items()}, least=2)


def test_attention(launches):
    """Every kernel's plan; the blocks of rows and keys cover the call; the
    workspace does not outgrow the tensors by more than the splits' sums."""
    calls = []
    for dt in (0, 1):
        for causal in (0, 1):
            for dim in (1, 33, 64, 72, 128):
                for b, q, k, h, kv, seqs in ((1, 1, 1, 1, 1, 0), (1, 1, 0, 4, 2, 0), (1, 1, 1 << 20, 28, 4, 0), (8, 1, 65536, 28, 4, 0),
                                             (1, 1, 1 << 24, 1, 1, 0), (2, 333, 333, 6, 2, 0), (1, 1 << 20, 1 << 20, 2, 1, 0),
                                             (1 << 20, 1, 1, 4, 4, 0), (1, 1 << 24, 5, 1, 1, 0), (64, 1, 333, 1 << 10, 1, 0),
                                             (1, 8192, 8192, 28, 4, 11), (1, 1 << 20, 1 << 20, 8, 1, 1 << 20), (1, 5, 5, 2, 2, 1),
                                             (1, 1 << 24, 1, 16, 16, 0), (1 << 20, 16, 1, 16, 1, 0), (1, 1 << 24, 1 << 24, 16, 16, 7)):
                    calls.append(["attention", b, q, k, h, kv, dim, seqs, causal, dt])
    found = launches(calls)
    check({c: ls for c, (ls, _) in found.items()}, least=3)
    for c, (ls, (fwd, bwd)) in found.items():
        _, b, q, k, h, kv, dim, seqs, causal, dt = json.loads(c)
        e, wide = (2 if dt else 4), -(-dim // 8) * 8
        tensors = (b * q * h * 4 + b * k * kv * 4) * (wide + 8) * e
        # sums of 512 splits of a few rows, of two blocks each of 512 stretches; lists
        assert fwd <= 2 * tensors + (1 << 20) + 512 * 128 * 4 * (128 * 2 + 2) * 4 + 16 * (b * q * h // 32 + seqs), c
        assert bwd <= 2 * tensors + b * q * h * 64 + (1 << 20) + 512 * 2 * 128 * 512 * 4 + 48 * (b * max(q * h, k) // 32 + seqs), c
