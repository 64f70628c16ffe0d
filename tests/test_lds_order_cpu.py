"""Exchanges between the lanes of a wave through shared memory are ordered in
the memory model, not only by today's instruction order (no GPU needed): in
the optimised device code of the token sort, every wave barrier stands between
wavefront fences, and both a write after other lanes' reads and a read after
another lane's write are so separated."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from muon_newton_schulz_06_amd import build  # noqa: E402


@pytest.fixture(scope="module")
def kernels():
    """{kernel: its lines that touch shared memory, fence or are barriers}."""
    cmd = [build.hipcc(), *build.flags(), "-emit-llvm", "-S", "--cuda-device-only", "-o", "-",
           os.path.join(build.CSRC, "embedding.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = {}
    for m in re.finditer(r"^define [^\n]*@(\w*embed_sort_\w+)\([^\n]*\n(.*?)^}", r.stdout, re.M | re.S):
        out[m.group(1)] = [t for t in m.group(2).splitlines()
                           if re.search(r"addrspace\(3\)|\bfence\b|wave\.barrier", t)]
    return out


def test_wave_barriers_are_fenced(kernels):
    seen = 0
    for name, lines in kernels.items():
        kinds = ["fence" if re.search(r'\bfence syncscope\("wavefront"\)', t) else
                 "barrier" if "wave.barrier" in t else
                 "access" if re.search(r"\b(load|store)\b", t) else "other" for t in lines]
        for i, k in enumerate(kinds):
            if k == "barrier":
                seen += 1
                assert kinds[i - 1] == "fence" and kinds[i + 1] == "fence", (name, lines[i - 1:i + 2])
    assert seen >= 2 * (1 + 4 + 16)  # two per round of the three small sorts alone


def test_counts_are_exchanged_in_order(kernels):
    """In a round the counts are read, then (fence) stored by one lane each,
    then (fence) read again."""
    for name, lines in kernels.items():
        if not any("wave.barrier" in t for t in lines):
            continue
        first, last = (f(i for i, t in enumerate(lines) if "wave.barrier" in t) for f in (min, max))
        kinds = "".join("b" if "wave.barrier" in t else "l" if re.search(r"\bload\b", t) else
                        "s" if re.search(r"\bstore\b", t) else "" for t in lines[first:last + 1])
        assert not re.search("ls|sl", kinds), (name, kinds)
