"""The norms with gradients as the package offers them outside a MoEBlock."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_block_norm import inputs

pytestmark = pytest.mark.gpu


def test_the_norm_after_the_last_block():
    """block_norm_autograd's weight and stream get their gradients: block_norm_bwd's bits."""
    moe = lib()
    d, up = inputs(33, 512, x="f32", branch=False)
    x, weight = d["x"].clone().requires_grad_(), d["weight"].clone().requires_grad_()
    r, h = moe.block_norm_autograd(x, weight)
    assert r is None
    h.backward(up["dh"])
    _, h0, stats = moe.block_norm(d["x"], d["weight"], save_for_backward=True)
    want = moe.block_norm_bwd(up["dh"], None, d["x"], stats, d["weight"])
    assert torch.equal(h, h0) and torch.equal(x.grad, want["dx"]) and torch.equal(weight.grad, want["d_weight"])
    moe.sync_status()


@pytest.mark.parametrize("gates", (1, 4, 20))
def test_every_operand(gates):
    moe = lib()
    d, up = inputs(20, 256, post="f32", gates=gates)
    leaves = {n: t.clone().requires_grad_() for n, t in d.items()}
    r, h = moe.block_norm_autograd(**leaves, residual_scale=0.7, branch_scale=0.5, eps=1e-5)
    torch.autograd.backward([r, h], [up["dr"], up["dh"]])
    how = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"], residual_scale=0.7, branch_scale=0.5)
    r0, h0, stats = moe.block_norm(d["x"], eps=1e-5, save_for_backward=True, **how)
    want = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **how)
    assert torch.equal(r, r0) and torch.equal(h, h0)
    for leaf, name in (("x", "dx"), ("branch", "d_branch"), ("weight", "d_weight"), ("post_weight", "d_post_weight"), ("gate", "d_gate")):
        assert torch.equal(leaves[leaf].grad, want[name])
    with torch.no_grad():
        assert moe.block_norm_autograd(**leaves)[0].grad_fn is None
    moe.sync_status()
