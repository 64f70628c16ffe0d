"""RMS norm over more rows than a grid dimension has workgroups for (2^32
threads): in place, 4.2 million rows of 4104 bf16 values (34 GB)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,dim", [((1 << 22) + 3, 4104), ((1 << 24) - 1, 1032)])
def test_rms_norm_many_rows(lib, tokens, dim):
    """Rows of one value each, 1 .. 8 in turn: y is their sign, rstd one over
    their size, both to a rounding (eps is 1e-6 of the smallest square)."""
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of free device memory")
    size = (torch.arange(tokens, device="cuda") % 8 + 1).to(torch.bfloat16)
    sign = torch.where(torch.arange(tokens, device="cuda") % 3 == 0, -1.0, 1.0).to(torch.bfloat16)
    x = torch.empty((tokens, dim), dtype=torch.bfloat16, device="cuda")
    x.copy_((size * sign)[:, None].expand(tokens, dim))
    y, _, rstd = lib.muon_rms_norm(x, torch.ones(dim, device="cuda"), eps=1e-6, out=x)
    assert y is x
    # half an ulp of the value for eps, the rest for dim + 8 fp32 roundings
    assert bool(((rstd * size.float() - 1).abs() <= 1e-6 + (dim + 8) * 2.0 ** -24).all())
    for lo in range(0, tokens, 1 << 20):
        part = x[lo:lo + (1 << 20)]
        assert bool((part == sign[lo:lo + (1 << 20), None]).all()), lo
    del x, y
    torch.cuda.empty_cache()
