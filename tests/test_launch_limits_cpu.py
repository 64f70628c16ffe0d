"""Launch sizes of the layer entry points at their documented limits (no GPU
needed): a stand-in for the runtime's launch, loaded ahead of it into a child
process, notes each launch and starts nothing.  A grid's dimension times the
workgroup's must stay below 2^32 threads, and a grid's second and third
dimensions at most 65535 workgroups."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STANDIN = r"""
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
typedef struct { uint32_t x, y, z; } dim3;
static dim3 grid, block;
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void* stream) { grid = g; block = b; return 0; }
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* lds, void** stream) {
  *g = grid; *b = block; *lds = 0; *stream = 0;
  return 0;
}
int hipGetDeviceCount(int* n) { *n = 1; return 0; }
int hipGetLastError(void) { return 0; }
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t lds, void* stream) {
  printf("%u %u %u %u %u %u\n", g.x, g.y, g.z, b.x, b.y, b.z);
  fflush(stdout);
  return 0;
}
"""

CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
A, B, C, D, E, F, G = (k << 50 for k in range(1, 8))
i64, f32, vp = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
big = ctypes.c_size_t(1 << 48)
def norm(tokens, dim, dt, res):
    return L.muon_rms_norm(vp(A), i64(dim), vp(B if res else 0), i64(dim), vp(C), 0, f32(1e-6), vp(A), i64(dim),
                           vp(B if res else 0), i64(dim), vp(F), i64(tokens), i64(dim), dt, None)
def norm_grad(tokens, dim, dt, res):
    return L.muon_rms_norm_grad(vp(A), i64(dim), vp(B), i64(dim), vp(C), 0, vp(F), None, i64(0), vp(A), i64(dim), vp(D),
                                0, i64(tokens), i64(dim), dt, vp(G), big, None)
def embed(tokens, dim, dt, res):
    return L.muon_embedding(vp(A), 8, i64(tokens), vp(B), i64(dim), i64(1 << 24), i64(dim), f32(1), vp(C), i64(dim), dt, None)
def embed_grad(tokens, dim, dt, res):
    return L.muon_embedding_grad(vp(A), i64(dim), vp(B), 8, i64(tokens), i64(1 << 24), i64(dim), f32(1), vp(C), i64(dim),
                                 dt, 0, 0, vp(G), big, None)
class Ffn(ctypes.Structure):
    _fields_ = [("n", i64 * 3), ("w", vp * 3), ("ld", i64 * 3), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32)]
class Grads(ctypes.Structure):
    _fields_ = [("p", vp * 4), ("ld", i64 * 4), ("dtype", ctypes.c_int32), ("acc", ctypes.c_int32)]
def ffn(tokens, model, dt, hidden):
    f = Ffn((tokens, model, hidden), (A, A + (1 << 49), B), (model, model, hidden), dt, 0)
    s = L.muon_gated_ffn(ctypes.byref(f), vp(C), i64(model), vp(D), i64(model), vp(E), big, vp(G), big, None)
    if s:
        return s
    W = B + (1 << 49)
    g = Grads((D, W, W + (1 << 46), W + (1 << 47)), (model, model, model, hidden), 0, 0)
    return L.muon_gated_ffn_grad(ctypes.byref(f), vp(C), i64(model), vp(F), i64(model), vp(E), big, ctypes.byref(g), vp(G),
                                 big, None)
for name, *args in json.loads(sys.argv[3]):
    print("call", json.dumps([name, *args]), flush=True)
    print("status", globals()[name](*args), flush=True)
"""

MEMORY = 288e9  # bytes of a GPU: what is larger cannot be called


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """{call: [(grid, block), ..]} of the calls given."""
    tmp = tmp_path_factory.mktemp("standin")
    src, so = tmp / "standin.c", tmp / "standin.so"
    src.write_text(STANDIN)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, src], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-c", CHILD, so, os.path.join(ROOT, "muon_newton_schulz_06_amd", "libmuon_ns.so"),
                            json.dumps(calls)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        out, call = {}, None
        for line in r.stdout.splitlines():
            if line.startswith("call "):
                call = line[5:]
                out[call] = []
            elif line.startswith("status "):
                assert line == "status 0", (call, line)
            else:
                n = [int(v) for v in line.split()]
                out[call].append((n[:3], n[3:]))
        return out
    return run


def rows_calls(name, tensors):
    """Every row length at both sides of the kernels' plans with as many tokens
    as the header allows and the memory holds (tensors: tokens × dim each)."""
    calls = []
    for dt, esz in ((0, 4), (1, 2)):
        for dim in (1, 64, 513, 1024, 1025, 4096, 4097, 4104, 8192, 16385, 32768, 65537, 1 << 20):
            fit = int(MEMORY / (tensors * dim * esz))
            for tokens in (1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, 1 << 23, 1 << 24, fit):
                if tokens <= min(fit, 1 << 24):
                    for res in (0, 1):
                        calls.append([name, tokens, dim, dt, res])
    return calls


def check(found, least=1):
    assert found
    for call, ls in found.items():
        assert len(ls) >= least, call
        for grid, block in ls:
            assert all(g >= 1 and b >= 1 for g, b in zip(grid, block)), (call, grid, block)
            assert all(g * b < 2 ** 32 for g, b in zip(grid, block)), (call, grid, block)
            assert grid[1] <= 65535 and grid[2] <= 65535, (call, grid, block)
            assert block[0] * block[1] * block[2] <= 1024, (call, grid, block)


@pytest.mark.parametrize("name", ["norm", "norm_grad", "embed", "embed_grad"])
def test_rows(launches, name):
    check(launches(rows_calls(name, 1)))


def test_norm_takes_every_row(launches):
    """As many row groups as tokens, whatever the grid's shape."""
    for call, ls in launches(rows_calls("norm", 1)).items():
        _, tokens, dim, dt, _ = json.loads(call)
        (grid, block), = ls
        chunks = -(-dim // (8 if dt else 4))
        per = 4 if block[0] == 256 and chunks <= (128 if dt else 256) else 1
        assert grid[0] * grid[1] * per >= tokens, call


def test_gated_ffn(launches):
    calls = []
    for dt, esz in ((0, 4), (1, 2)):
        for model, hidden in ((1, 1), (64, 64), (64, 1 << 20), (1 << 20, 64), (3584, 18944), (8192, 32768), (20001, 20001)):
            # x, y, dx, dy; h, dg, du; a and b; weights and gradients
            fit = int((MEMORY - 3 * model * hidden * (esz + 4)) / (4 * model * esz + 3 * hidden * esz + 8 * hidden))
            for tokens in (1, 33, 64, 65, 1 << 14, 1 << 20, 1 << 24, fit):
                if 1 <= tokens <= min(fit, 1 << 24):
                    calls.append(["ffn", tokens, model, dt, hidden])
    check(launches(calls), least=5)
