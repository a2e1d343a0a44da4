"""A block around the layer (MoEBlock): norms, layer, gate and residual as they
are used together, in training with clipped gradients and in a decode step."""
import math

import pytest
import torch

from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu

H, E, K, I = 256, 16, 4, 128


def make(moe, seed=0, routing=None, **kw):
    g = torch.Generator().manual_seed(seed)
    layer = moe.MoELayer(H, E, K, I, device=dev(), routing=routing)
    block = moe.MoEBlock(layer, **kw)
    with torch.no_grad():
        layer.w_router.copy_(torch.randn((H, E), generator=g) * H ** -0.5)
        layer.gate_up.copy_(torch.randn(layer.gate_up.shape, generator=g) * H ** -0.5)
        layer.down.copy_(torch.randn(layer.down.shape, generator=g) * I ** -0.5)
        for n in ("norm", "post_norm", "scale"):
            v = getattr(block, n)
            if v is not None:
                v.copy_(1.0 + 0.2 * torch.randn(H, generator=g))
    return block


def stream(T, t, seed=1):
    return (2.0 * torch.randn((T, H), generator=torch.Generator().manual_seed(seed + T))).to(t).to(dev())


KINDS = (dict(), dict(post_norm=True), dict(learned_scale=1.0, residual_scale=0.7), dict(post_norm=True, learned_scale=0.5, branch_scale=0.22))


@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("t", (torch.float32, torch.bfloat16))
def test_a_block_is_its_steps(kw, t):
    """Forward and gradients bit for bit those of the operators called one by one."""
    moe = lib()
    block, x = make(moe, **kw), stream(77, t).requires_grad_()
    following = torch.linspace(0.5, 1.5, H, device=dev()).requires_grad_()
    r, h = block(x, next_norm=following)
    dr, dh = stream(77, t, 5), stream(77, torch.bfloat16, 6)
    torch.autograd.backward([r, h], [dr, dh])
    p = [v.detach() for v in (block.layer.w_router, block.layer.gate_up, block.layer.down)]
    x0, gate = x.detach(), None if block.scale is None else block.scale.detach().unsqueeze(0)
    around = dict(weight=following.detach(), post_weight=None if block.post_norm is None else block.post_norm.detach(), gate=gate,
                  residual_scale=block.residual_scale, branch_scale=block.branch_scale)
    _, h0, s0 = moe.block_norm(x0, block.norm.detach(), save_for_backward=True)
    y, st = moe.moe_forward(h0, *p, K, save_for_backward=True)
    r1, h1, s1 = moe.block_norm(x0, branch=y, save_for_backward=True, **around)
    assert torch.equal(r, r1) and torch.equal(h, h1)
    g1 = moe.block_norm_bwd(dh, dr, x0, s1, branch=y, **around)
    gl = moe.moe_backward(g1["d_branch"], st, *p, want_dw_router=True)
    g0 = moe.block_norm_bwd(gl["dx"], None, x0, s0, block.norm.detach())
    want = {x: g1["dx"] + g0["dx"], block.norm: g0["d_weight"], following: g1["d_weight"], block.layer.w_router: gl["d_w_router"],
            block.layer.gate_up: gl["d_gate_up"], block.layer.down: gl["d_down"]}
    if block.post_norm is not None:
        want[block.post_norm] = g1["d_post_weight"]
    if block.scale is not None:
        want[block.scale] = g1["d_gate"][0]
    for leaf, grad in want.items():
        assert torch.equal(leaf.grad, grad)
    moe.sync_status()


def test_against_a_model():
    """The block and its gradients against autograd in 64 bits, at the block's
    own choice of experts.  Some 16 roundings to bf16 lie on a path, each of at
    most 2^-8 of what it rounds."""
    moe = lib()
    block, x = make(moe, post_norm=True, learned_scale=0.5), stream(50, torch.float32).requires_grad_()
    r, _ = block(x)
    dr = stream(50, torch.float32, 9)
    r.backward(dr)
    h = moe.block_norm(x.detach(), block.norm.detach())[1]
    ids, _ = moe.route(h, block.layer.w_router.detach(), K)
    leaves = [x] + list(block.parameters())
    names = {id(p): n for n, p in block.named_parameters()}
    v = {id(p): p.detach().double().requires_grad_() for p in leaves}
    at = lambda p: v[id(p)]

    def rms(t, w):
        return t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-6) * w

    hx = rms(at(x), at(block.norm))
    z = (hx @ at(block.layer.w_router)).gather(1, ids.long())
    w = torch.softmax(z, 1)
    G, D = at(block.layer.gate_up).view(E, H, 2 * I), at(block.layer.down).view(E, I, H)
    y = torch.zeros_like(hx)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        u = hx[t] @ G[e]
        y = y.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ D[e]))
    ref = at(x) + at(block.scale) * rms(y, at(block.post_norm))
    ref.backward(dr.double())

    def near(name, got, want):
        assert float((got.double() - want).norm()) <= 16 * 2.0 ** -8 * float(want.norm()), name

    near("r", r.detach(), ref.detach())
    for p in leaves:
        near(names.get(id(p), "x"), p.grad, at(p).grad)


def test_a_run_of_blocks_and_a_training_step():
    """Three blocks, each block's end fused with the next one's norm: the same
    bits as norms of their own, and a step with clipped gradients."""
    moe = lib()
    blocks = torch.nn.ModuleList(make(moe, i, post_norm=i == 1) for i in range(3))
    x = stream(90, torch.float32)

    def run(fused):
        blocks.zero_grad(set_to_none=True)
        r, h = x, None
        for i, b in enumerate(blocks):
            following = blocks[i + 1].norm if fused and i < 2 else None
            r, h = b(r, h, next_norm=following)
            if not fused:
                h = None
        r.square().mean().backward()
        return r.detach(), [p.grad.clone() for p in blocks.parameters()]

    fused, grads = run(True)
    plain, more = run(False)
    assert torch.equal(fused, plain)      # fp32 stream: the norm sees the same r
    # the gradient of a stream's norm joins dr in one kernel or in two: fp32 roundings of the stream, and bf16 ones that follow from them
    for a, b in zip(grads, more):
        assert float((a.double() - b.double()).norm()) <= 2.0 ** -6 * float(b.double().norm())
    want = math.sqrt(sum(float(g.double().square().sum()) for g in more))
    norm = moe.clip_grad_norm(blocks.parameters(), 0.5 * want)
    assert abs(float(norm) - want) <= 2.0 ** -17 * want
    after = math.sqrt(sum(float(p.grad.double().square().sum()) for p in blocks.parameters()))
    assert abs(after - 0.5 * want) <= 2.0 ** -8 * want
    twice = list(blocks.parameters()) * 2
    assert abs(float(moe.clip_grad_norm(twice, 1e9)) - after) <= 2.0 ** -17 * after
    blocks.zero_grad(set_to_none=True)
    with pytest.raises(ValueError):
        moe.clip_grad_norm(blocks.parameters(), 1.0)
    moe.sync_status()


@pytest.mark.parametrize("routing", (None, dict(score="sigmoid", n_groups=4, top_groups=2, scale=2.5), dict(renorm=False)), ids=str)
def test_decode(routing):
    """Few tokens through a run of blocks: near the training path's values (a
    rounding of the experts' products apart), and the operators' bits."""
    moe = lib()
    how = None if routing is None else moe.Routing(**routing)
    blocks = [make(moe, i, routing=how) for i in range(2)]
    x = stream(12, torch.bfloat16)
    r, h = blocks[0].decode(x, next_norm=blocks[1].norm)
    r, _ = blocks[1].decode(r, h)
    with torch.no_grad():
        a, b = blocks[0](x, next_norm=blocks[1].norm)
        a, _ = blocks[1](a, b)
    assert not r.requires_grad
    assert float((r.double() - a.double()).norm()) <= 16 * 2.0 ** -8 * float(a.double().norm())
    layer = blocks[0].layer
    h0 = moe.block_norm(x, blocks[0].norm.detach())[1]
    bias = None if how is None else layer.balance_bias
    y, ids, w = moe.moe_forward_few(h0, layer.w_router.detach(), layer.gate_up.detach(), layer.down.detach(), K, routing=how, balance_bias=bias)
    assert torch.equal(layer.decode(h0), y)
    graph = moe.DecodeGraph(12, layer.w_router.detach(), moe.BF16Experts(layer.gate_up.detach(), layer.down.detach(), E), K, routing=how,
                            balance_bias=bias)
    assert torch.equal(graph(h0), y) and torch.equal(graph.ids, ids) and torch.equal(graph.w, w)
    graph.refresh_router_split()
    assert torch.equal(graph(2 * h0), layer.decode(2 * h0))
    moe.sync_status()


def test_gate_of_each_sequence():
    moe = lib()
    block, x = make(moe), stream(60, torch.bfloat16).requires_grad_()
    gate = torch.randn((3, H), device=dev(), dtype=torch.bfloat16, requires_grad=True)
    r, h = block(x, gate=gate)
    assert h is None
    r.float().square().mean().backward()
    assert gate.grad.shape == gate.shape and bool(gate.grad.isfinite().all()) and float(gate.grad.abs().max()) > 0
    # a row's output is that of its own sequence alone
    with torch.no_grad():
        for i in range(3):
            one, _ = block(x[20 * i:20 * i + 20], gate=gate[i:i + 1])
            assert torch.equal(one, r[20 * i:20 * i + 20])
    with pytest.raises(ValueError):
        make(moe, learned_scale=1.0)(x, gate=gate)


def test_only_some_operands_ask_for_gradients():
    """An unused output, frozen operands, and no gradient at all."""
    moe = lib()
    from token_dispatch_grouped_softmax_gb300.layer import block_norm

    x, y = stream(9, torch.float32), stream(9, torch.bfloat16, 3)
    w = torch.ones(H, device=dev(), requires_grad=True)
    r, h = block_norm(x, w, y)
    r.sum().backward()
    assert w.grad is not None and bool((w.grad == 0).all())     # h was not used
    w.grad = None
    r, h = block_norm(x, w, y)
    h.float().sum().backward()
    assert x.grad is None and float(w.grad.abs().max()) > 0
    with torch.no_grad():
        assert block_norm(x, w, y)[1].grad_fn is None
    assert block_norm(x, w.detach(), y)[0].grad_fn is None
    strided = y.t().contiguous().t()                             # made contiguous by the module's function
    assert torch.equal(block_norm(x, w.detach(), strided)[0], block_norm(x, w.detach(), y)[0])


def test_refusals():
    moe = lib()
    block = make(moe)
    experts = moe.BF16Experts(block.layer.gate_up.detach(), block.layer.down.detach(), E)
    with pytest.raises(ValueError):
        moe.DecodeGraph(4, block.layer.w_router.detach(), experts, K, bf16_rows=48)
    with pytest.raises(ValueError):
        moe.DecodeGraph(4, block.layer.w_router.detach()[:, :8].contiguous(), experts, K)
    with pytest.raises(moe.MoEError):
        block.decode(stream(129, torch.bfloat16))
    with pytest.raises((ValueError, TypeError)):
        block.decode(stream(4, torch.float16))
