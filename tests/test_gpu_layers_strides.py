"""The modules on inputs and incoming gradients of any strides: the bits they
give for the same values in contiguous rows."""
import pytest
import torch

from test_gpu_layers import DTYPES, rand

pytestmark = pytest.mark.gpu

LAYOUTS = {
    "transposed": lambda s, t: rand((24, 40), s, t).cuda().t(),
    "every second": lambda s, t: rand((40, 48), s, t).cuda()[:, ::2],
    "one row for all": lambda s, t: rand((24,), s, t).cuda().expand(40, 24),
    "3-D, every second": lambda s, t: rand((5, 8, 48), s, t).cuda()[..., ::2],
    "3-D, transposed": lambda s, t: rand((8, 5, 24), s, t).cuda().transpose(0, 1),
    "3-D, columns first": lambda s, t: rand((24, 40), s, t).cuda().t().unflatten(0, (5, 8)),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_modules(lib, layout, dtype):
    torch.manual_seed(4)
    make = LAYOUTS[layout]
    ffn = lib.GatedFFN(24, 40, device="cuda", dtype=dtype)
    norm = lib.RMSNorm(24, device="cuda", dtype=dtype)
    emb = lib.Embedding(9, 24, device="cuda", dtype=dtype)
    params = [*ffn.parameters(), *norm.parameters(), *emb.parameters()]

    def run(copy):
        x, r, dy, ds = (make(k, dtype) for k in range(4))
        if copy:
            x, r, dy, ds = (t.contiguous() for t in (x, r, dy, ds))
        ids = torch.arange(x.numel() // 24, device="cuda").reshape(x.shape[:-1]) % 9
        x, r = x.detach().requires_grad_(), r.detach().requires_grad_()
        y, s = norm(x, r)
        outs = [ffn(x), y, s, emb(ids)]
        grads = torch.autograd.grad(outs, [x, r, *params], [dy, ds, dy, ds])
        return [t.detach() for t in (*outs, *grads)]
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
