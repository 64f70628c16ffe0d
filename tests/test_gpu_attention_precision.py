"""The attention of bf16 tensors to the precision that its roundings leave
(tolerances and cases: test_attention_precision_cpu.py, where each of the choices
that they rest on is taken back in a model and found)."""
import pytest
import torch

from test_attention_precision_cpu import CASES, errors, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CASES)
def test_precision(lib, name):
    ts = inputs(name)
    do, q, k, v, lam, offsets = ts
    do, q, k, v = (torch.from_numpy(t).bfloat16().cuda() for t in (do, q, k, v))
    lam, kw = torch.from_numpy(lam).float().cuda(), {}
    if offsets is not None:
        do, q, k, v, kw = do[0], q[0], k[0], v[0], dict(offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    out, saved = lib.muon_diff_attention(q, k, v, lam, save=True, **kw)
    dq, dk, dv, _ = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, **kw)
    got = dict(out=out, dq=dq, dk=dk, dv=dv)
    got = {n: (t if offsets is None else t[None]).double().cpu().numpy() for n, t in got.items()}
    found = errors(got, name, ts)
    print(name, {n: round(float(e), 3) for n, e in found.items()}, flush=True)
    assert max(found.values()) <= 1.0, found
