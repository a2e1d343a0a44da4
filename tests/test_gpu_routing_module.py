"""MoELayer with a Routing where no gradient is asked for."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_routing_layer import layer_inputs

pytestmark = pytest.mark.gpu

T, H, E, K_TOKEN, I = 90, 128, 16, 4, 64


def module(moe, d, **kw):
    layer = moe.MoELayer(H, E, K_TOKEN, I, device=dev(), **kw)
    with torch.no_grad():
        layer.w_router.copy_(d["wr"])
        layer.gate_up.copy_(d["gate_up"])
        layer.down.copy_(d["down"])
    return layer


@pytest.mark.parametrize("routing", (dict(renorm=False), dict(score="sigmoid", n_groups=4, top_groups=2, scale=2.5)))
def test_inference(routing):
    """Under no_grad, and with parameters that need no gradient, every Routing
    runs, keeps nothing for a backward, counts the loads and gives
    moe_forward's bits; the same where the layer trains, which a dense
    gradient does not."""
    moe = lib()
    d = layer_inputs(4, T, H, E, I)
    how = moe.Routing(**routing)
    layer = module(moe, d, routing=how)
    with torch.no_grad():
        layer.balance_bias.copy_(d["bias"])
    want, st = moe.moe_forward(d["x"], d["wr"], d["gate_up"], d["down"], K_TOKEN, routing=how, balance_bias=d["bias"])
    with torch.no_grad():
        y = layer(d["x"])
    assert torch.equal(y, want) and y.grad_fn is None and torch.equal(layer.last_counts, st.counts)
    if how.dense_gradient:
        with pytest.raises(ValueError, match="dX"):
            layer(d["x"])
    else:
        assert torch.equal(layer(d["x"]).detach(), want)
    layer.last_counts = None
    layer.requires_grad_(False)
    y = layer.eval()(d["x"])
    assert torch.equal(y, want) and y.grad_fn is None and torch.equal(layer.last_counts, st.counts)
    before = layer.balance_bias.clone()
    layer.update_balance_bias(0.5)
    assert torch.equal(layer.balance_bias, moe.route_balance_bias(before, st.counts, 0.5))
    moe.sync_status()


def test_without_a_balance_bias():
    """balance=False: no bias, and the choice that moe_forward makes without one,
    by the logits: logits whose scores round to the same value keep their order."""
    moe = lib()
    d = layer_inputs(5, T, H, E, I)
    d["x"][:, 0] = 2.0
    d["wr"][:, :] *= 0.01
    d["wr"][0] = 10.0 + 2.0 ** -8 * torch.arange(E, device=dev())   # logits of 20 and more: every sigmoid is 1
    how = moe.Routing(score="sigmoid")
    layer = module(moe, d, routing=how, balance=False)
    want, st = moe.moe_forward(d["x"], d["wr"], d["gate_up"], d["down"], K_TOKEN, routing=how)
    assert bool((st.ids > 7).all())                                 # equal scores would take the lowest experts
    assert torch.equal(layer(d["x"]).detach(), want)
    assert "balance_bias" not in dict(layer.named_buffers())
    with pytest.raises(ValueError):
        layer.update_balance_bias(0.1)
    with torch.no_grad():
        assert torch.equal(layer(d["x"]), want)
    with pytest.raises(ValueError):
        moe.MoELayer(H, E, K_TOKEN, I, device=dev(), balance=False)
    moe.sync_status()
