"""The layer with a Routing, and the layer with 4-bit experts, as a program
calls them: whole forward and backward against a 64-bit model by autograd,
and against the same steps called one by one."""
import numpy as np
import pytest
import torch

import ref_select as ref
from gpu_helpers import dev, f64, lib, npi
from parity import assert_close

pytestmark = pytest.mark.gpu


def layer_inputs(seed, T, H, E, I):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s, scale=1.0: (scale * torch.randn(s, generator=g)).bfloat16().to(dev())
    return dict(x=bf(T, H), dy=bf(T, H), gate_up=bf(E * H, 2 * I, scale=H ** -0.5), down=bf(E * I, H, scale=I ** -0.5),
                wr=(torch.randn((H, E), generator=g) * H ** -0.5).to(dev()),
                bias=(0.1 * torch.randn(E, generator=g)).to(dev()))


def model64(d, ids, routing, I):
    """y and the gradients of x, W_r, gate_up, down for the given choice, in 64 bits by autograd."""
    H, E = d["wr"].shape
    x, wr, gu, dn = (d[n].double().cpu().requires_grad_() for n in ("x", "wr", "gate_up", "down"))
    z = x @ wr
    s = torch.sigmoid(z) if routing.score == "sigmoid" else torch.softmax(z, 1)
    p = s.gather(1, ids)
    w = routing.scale * (p / p.sum(1, keepdim=True) if routing.renorm else p)
    G, D = gu.view(E, H, 2 * I), dn.view(E, I, H)
    y = torch.zeros_like(x)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            u = x[t] @ G[e]
            y = y.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ D[e]))
    y.backward(d["dy"].double().cpu())
    return y, x.grad, wr.grad, gu.grad, dn.grad


@pytest.mark.parametrize("kw", [dict(score="sigmoid", n_groups=4, top_groups=2, scale=2.5),
                                dict(score="sigmoid", renorm=False), dict(n_groups=2, top_groups=1, group_score="max")])
def test_layer_with_routing_trains(kw):
    """Forward and gradients of MoELayer with a Routing and a balance bias, and the bias's update."""
    moe = lib()
    T, H, E, k, I = 150, 128, 16, 4, 64
    d = layer_inputs(3, T, H, E, I)
    routing = moe.Routing(**kw)
    layer = moe.MoELayer(H, E, k, I, device=dev(), routing=routing)
    with torch.no_grad():
        layer.w_router.copy_(d["wr"])
        layer.gate_up.copy_(d["gate_up"])
        layer.down.copy_(d["down"])
        layer.balance_bias.copy_(d["bias"])
    x = d["x"].clone().requires_grad_()
    y = layer(x)
    y.backward(d["dy"])
    moe.sync_status()
    ids, _ = routing.select(moe.route_logits(d["x"], d["wr"]), k, d["bias"])
    y64, dx, dwr, dgu, ddn = (t.detach().numpy() for t in model64(d, ids.long().cpu(), routing, I))
    r = ref.select(f64(d["x"]) @ f64(d["wr"]), k, bias=f64(d["bias"]), **kw)
    same = (npi(ids) == r["ids"]).all(1)
    assert (same | (r["gap"] < 1e-5)).all()
    assert_close("y (routing)", f64(y.detach()), y64)
    assert_close("dX (routing)", f64(x.grad), dx)
    assert_close("d_W_r (routing)", f64(layer.w_router.grad), dwr, bf16_out=False)
    assert_close("d_gate_up (routing)", f64(layer.gate_up.grad), dgu, operand_abs=np.abs(dgu) + np.abs(dgu).max())
    assert_close("d_down (routing)", f64(layer.down.grad), ddn, operand_abs=np.abs(ddn) + np.abs(ddn).max())
    n = np.bincount(npi(ids).ravel(), minlength=E)
    np.testing.assert_array_equal(npi(layer.last_counts), n)
    want = d["bias"].cpu().numpy() + np.float32(0.01) * np.sign(n.sum() - E * n).astype(np.float32)
    layer.update_balance_bias(0.01)
    np.testing.assert_array_equal(layer.balance_bias.cpu().numpy(), want)


def test_routing_refusals():
    moe = lib()
    d = layer_inputs(1, 8, 64, 8, 64)
    args = (d["x"], d["wr"], d["gate_up"], d["down"], 2)
    with pytest.raises(ValueError):   # a dense gradient
        moe.moe_forward(*args, save_for_backward=True, routing=moe.Routing(renorm=False))
    moe.moe_forward(*args, routing=moe.Routing(renorm=False))
    with pytest.raises(ValueError):   # a balance bias without a Routing
        moe.moe_forward(*args, balance_bias=d["bias"])
    with pytest.raises(ValueError):
        moe.MoELayer(64, 8, 2, 64, device=dev()).update_balance_bias(0.1)
    with pytest.raises(ValueError):
        moe.moe_forward_w4(d["x"], d["wr"][:, :4].contiguous(), moe.W4Experts.quantize(d["gate_up"], d["down"], 8, 64), 2)
    moe.sync_status()


def test_a_plain_routing_is_the_router():
    """Softmax, one group, renormalised: the ids of ops.route, and its weights
    to the last places (the same quotients, summed in another order)."""
    moe = lib()
    d = layer_inputs(2, 300, 128, 32, 64)
    args = (d["x"], d["wr"], d["gate_up"], d["down"], 4)
    y0, st0 = moe.moe_forward(*args)
    y1, st1 = moe.moe_forward(*args, routing=moe.Routing())
    assert torch.equal(st0.ids, st1.ids)
    np.testing.assert_allclose(f64(st1.w), f64(st0.w), rtol=16 * 2 * ref.U)
    assert_close("y (plain Routing)", f64(y1), f64(y0))


@pytest.mark.parametrize("T", (1, 7, 64, 400))
@pytest.mark.parametrize("zeros", (False, True))
def test_w4_layer(T, zeros):
    """moe_forward_w4 with a shared expert against the 64-bit layer on the
    decoded weights: a decode batch, and one large enough (400 tokens, 100
    rows an expert) for the bf16 grouped GEMMs."""
    moe = lib()
    H, E, k, I, group = 256, 8, 2, 128, 64
    d = layer_inputs(T, T, H, E, I)
    s = layer_inputs(T + 1, T, H, 1, 192)
    experts = moe.W4Experts.quantize(d["gate_up"], d["down"], E, group, zeros)
    shared = moe.W4Experts.quantize(s["gate_up"], s["down"], 1, group, zeros)
    routing = moe.Routing(score="sigmoid", n_groups=4, top_groups=2, scale=2.5)
    y, ids, w = moe.moe_forward_w4(d["x"], d["wr"], experts, k, shared=shared, routing=routing, balance_bias=d["bias"])
    moe.sync_status()
    x = f64(d["x"])
    back = [f64(ref_w) for ref_w in experts.dequantize() + shared.dequantize()]
    # scale * (code - zero) rounded to bf16 is what the large path multiplies; the decode path has it exact
    exact = []
    for (q, sc, z), K, n in ((experts.gate_up, H, 0), (experts.down, I, 1), (shared.gate_up, H, 2), (shared.down, 192, 3)):
        W = ref.unpack(npi(q), f64(sc), None if z is None else npi(z), K, q.shape[1], group)
        np.testing.assert_allclose(back[n].reshape(W.shape), W, rtol=2.0 ** -8)
        exact.append(W)
    ids, w = npi(ids), f64(w)
    gu, _ = ref.experts(np.repeat(x[:, None], k, 1), ids, exact[0])
    p, _ = ref.experts(ref.silu(gu[..., :I]) * gu[..., I:], ids, exact[1])
    gs, _ = ref.experts(x[:, None], np.zeros((T, 1), int), exact[2])
    ps, _ = ref.experts(ref.silu(gs[..., :192]) * gs[..., 192:], np.zeros((T, 1), int), exact[3])
    assert_close("y (4-bit, T %d)" % T, f64(y), (p * w[..., None]).sum(1) + ps[:, 0])


def test_decode_graph():
    """One capture, several batches and routings, W_r changed and refreshed: the bits of the plain call."""
    moe = lib()
    T, H, E, k, I = 5, 256, 16, 4, 128
    d = layer_inputs(7, T, H, E, I)
    experts = moe.W4Experts.quantize(d["gate_up"], d["down"], E, 64)
    routing = moe.Routing(score="sigmoid", n_groups=4, top_groups=2)
    g = moe.DecodeGraph(T, d["wr"], experts, k, routing=routing, balance_bias=d["bias"])
    for seed in range(3):
        x = layer_inputs(20 + seed, T, H, E, I)["x"]
        y = g(x).clone()
        want, ids, w = moe.moe_forward_w4(x, d["wr"], experts, k, routing=routing, balance_bias=d["bias"])
        assert torch.equal(y, want) and torch.equal(g.ids, ids) and torch.equal(g.w, w)
        d["wr"].mul_(-1.0)
        g.refresh_router_split()
    moe.sync_status()
