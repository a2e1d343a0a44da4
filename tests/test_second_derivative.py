"""The layer's and the norms' gradients are first derivatives: differentiating
them again raises, and everything else of create_graph=True works."""
import pytest
import torch


def square():
    """x -> x^2 with a backward that records no graph, as the kernels' do."""
    from token_dispatch_grouped_softmax_gb300 import layer

    class Square(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, n):
            ctx.save_for_backward(x)
            return x * x

        @staticmethod
        @layer._first_order
        def backward(ctx, d):
            return 2 * ctx.saved_tensors[0] * d, None

    return lambda x: Square.apply(x, 2)


@pytest.mark.parametrize("loss", (lambda y: y.sum(), lambda y: (y * y).sum()), ids=("linear", "square"))
def test_refused(loss):
    """Also where the incoming gradient has no graph of its own."""
    x = torch.tensor([1.0, -2.0, 3.0], requires_grad=True)
    total = loss(square()(x))
    g, = torch.autograd.grad(total, x, create_graph=True)
    plain, = torch.autograd.grad(loss(x * x), x)
    assert torch.equal(g.detach(), plain)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (loss(square()(x)) + (g * g).sum()).backward()     # a penalty on the gradient beside the loss


def test_first_derivatives_are_as_before():
    x = torch.tensor([1.0, -2.0], requires_grad=True)
    g, = torch.autograd.grad(square()(x).sum(), x)
    assert not g.requires_grad and g.tolist() == [2.0, -4.0]
    square()(x).sum().backward(create_graph=True)
    assert x.grad.tolist() == [2.0, -4.0]


@pytest.mark.gpu
@pytest.mark.parametrize("what", ("norm", "layer", "routed layer", "block"))
@pytest.mark.parametrize("linear", (True, False))
def test_on_the_gpu(what, linear):
    from gpu_helpers import dev, lib

    moe = lib()
    H = 64
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, H), generator=g).to(torch.bfloat16).to(dev()).requires_grad_()
    layer = moe.MoELayer(H, 8, 2, 64, device=dev(), routing=moe.Routing() if what == "routed layer" else None)
    with torch.no_grad():
        for p in layer.parameters():
            p.copy_(0.1 * torch.randn(p.shape, generator=g))
    weight = torch.ones(H, device=dev(), requires_grad=True)
    if what == "norm":
        run = lambda: moe.BlockNormFunction.apply(x, weight, None, None, None, 1.0, 1.0, 1e-6)[1]
    elif what == "block":
        block = moe.MoEBlock(layer)
        run = lambda: block(x)[0]
    else:
        run = lambda: layer(x)
    loss = lambda: run().float().sum() if linear else run().float().square().sum()
    plain, = torch.autograd.grad(loss(), x)
    d, = torch.autograd.grad(loss(), x, create_graph=True)
    assert not plain.requires_grad and torch.equal(d.detach(), plain)
    with pytest.raises(RuntimeError, match="differentiated again"):
        d.float().square().sum().backward()
    moe.sync_status()
