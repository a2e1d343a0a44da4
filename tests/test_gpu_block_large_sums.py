"""The sums over columns and the gates' gradients of a block's norms beyond
2^31 elements, element by element.  Tolerances as in test_gpu_block_norm, for
the rows that are not zero: zeros add nothing to a sum."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_block_norm import check, model, sizes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gates", (1, 10, 270000))
def test_sums_beyond_2_31_elements(gates):
    moe = lib()
    T, H, tail = 270000, 8192, 3
    g = torch.Generator(device=dev()).manual_seed(1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=dev())
    branch, dh, dr = (torch.zeros_like(x) for _ in range(3))
    for t in (x, branch, dh, dr):
        t[-tail:] = torch.randn((tail, H), generator=g, device=dev()).to(torch.bfloat16)
    weight = 1 + 0.1 * torch.randn(H, generator=g, device=dev())
    gate = torch.ones((gates, H), dtype=torch.bfloat16, device=dev())
    gate[-tail:] = 0.5
    stats = moe.block_norm(x, weight, branch, gate=gate, save_for_backward=True)[2]
    grads = moe.block_norm_bwd(dh, dr, x, stats, weight, branch, gate=gate)
    moe.sync_status()
    own = gates == T
    mine = tail if own else 1      # gates of the last rows
    d = dict(x=x[-tail:], branch=branch[-tail:], weight=weight, post_weight=None, gate=gate[-mine:])
    up = dict(dh=dh[-tail:], dr=dr[-tail:])
    v, r64, h64 = model(d, 1.0, 1.0)
    torch.autograd.backward([r64, h64], [up["dr"].double(), up["dh"].double()])
    size = sizes(d, up, 1.0, 1.0)
    check("d_weight", grads["d_weight"], v["weight"].grad, size["d_weight"], tail)
    check("d_gate", grads["d_gate"][-mine:], v["gate"].grad, size["d_gate"], tail)
    check("dx", grads["dx"][-tail:], v["x"].grad, size["dx"])
    check("d_branch", grads["d_branch"][-tail:], v["branch"].grad, size["d_branch"])
    if 1 < gates < T:
        assert bool((grads["d_gate"][:-1] == 0).all())
    if own:     # a row's gate alone: the bits of a call on the last rows
        rows = [t[-tail:].contiguous() for t in (x, branch, dh, dr, gate)]
        st = moe.block_norm(rows[0], weight, rows[1], gate=rows[4], save_for_backward=True)[2]
        some = moe.block_norm_bwd(rows[2], rows[3], rows[0], st, weight, rows[1], gate=rows[4])
        assert torch.equal(grads["d_gate"][-tail:], some["d_gate"])
        assert all(bool((grads["d_gate"][i:i + 30000] == 0).all()) for i in range(0, T - tail - 30000, 30000))
        assert bool((grads["d_gate"][-tail - 30000:-tail] == 0).all())
    assert float(v["gate"].grad.abs().median()) > 0.1      # what is compared is not small
