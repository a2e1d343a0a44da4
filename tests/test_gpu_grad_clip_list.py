"""Clipping: factors at the edge of its two steps, gradients of any dense
layout, and the version counters of what is written.  Tolerances as in
test_gpu_grad_clip."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_grad_clip import NORM

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("small", (2.0 ** 51, 2.0 ** 52, 2.0 ** 53, 2.0 ** 60, 0.0))
@pytest.mark.parametrize("t", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("inplace", (False, True))
def test_a_factor_around_2_to_the_minus_64(small, t, inplace):
    """A norm of 2^64 and a little more: the factor is 2^-64 but for a rounding, and its first step 1."""
    moe = lib()
    grads = [torch.tensor([2.0 ** 64, small, -2.0 ** 40], device=dev()).to(t)]
    norm64 = float(grads[0].double().norm())
    want = grads[0].double() / norm64
    out = grads if inplace else [torch.zeros_like(grads[0])]
    norm = moe.clip_grads(grads, 1.0, out=out)
    assert abs(float(norm) - norm64) <= NORM * norm64
    half = torch.finfo(t).eps / 2
    assert bool(((out[0].double() - want).abs() <= (2 * NORM + half) * want.abs()).all()), out[0]


def test_what_is_written_has_a_new_version():
    """A tensor that autograd keeps for a backward and that a call then writes is noticed there."""
    moe = lib()
    a, b = torch.ones(8, device=dev()), torch.ones(8, device=dev())
    for call, out in ((lambda: moe.clip_grads([a], 1.0), a), (lambda: moe.clip_grads([a], 1.0, out=[b]), b)):
        leaf = torch.ones(8, device=dev(), requires_grad=True)
        y = (leaf * out).sum()
        version = out._version
        call()
        assert out._version > version
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    version = a._version
    moe.clip_grads([a], 1.0, out=[b])
    moe.grad_norm([a])
    assert a._version == version          # only read
    x = torch.ones((1, 64), dtype=torch.bfloat16, device=dev())
    gate_up, down = torch.ones((64, 128), dtype=torch.bfloat16, device=dev()), torch.ones((64, 64), dtype=torch.bfloat16, device=dev())
    y = torch.zeros_like(x)
    version = y._version
    moe.experts_few(x, torch.zeros((1, 1), dtype=torch.int32, device=dev()), torch.ones((1, 1), device=dev()), gate_up, down, out=y)
    assert y._version > version
    bias = torch.zeros(4, device=dev())
    version = bias._version
    moe.route_balance_bias(bias, torch.ones(4, dtype=torch.int32, device=dev()), 0.1, out=bias)
    assert bias._version > version
    with torch.inference_mode():
        kept = [torch.full((4,), 2.0, device=dev())]
        moe.clip_grads(kept, 1.0)
    moe.clip_grads(kept, 1.0)             # an inference tensor has no version, and is scaled as before
    assert float(kept[0].norm()) <= 1.0 + 1e-5
    moe.sync_status()


LAYOUTS = {"transposed": ((96, 40), lambda t: t.t()), "odd transposed": ((33, 7), lambda t: t.t()), "permuted": ((5, 6, 7), lambda t: t.permute(2, 0, 1)),
           "channels last": ((3, 8, 5, 4), lambda t: t.to(memory_format=torch.channels_last)), "sizes of one": ((1, 9, 1), lambda t: t.permute(2, 1, 0))}


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("t", (torch.float32, torch.bfloat16))
def test_dense_layouts(name, t):
    """A gradient has its parameter's strides, whatever they are."""
    moe = lib()
    shape, layout = LAYOUTS[name]
    g = torch.Generator(device=dev()).manual_seed(3)
    first = torch.randn(shape, generator=g, device=dev()).to(t)
    grads = [layout(first), torch.randn((50,), generator=g, device=dev()).to(t)]
    want = float(sum(v.double().square().sum() for v in grads).sqrt())
    refs = [v.double() / (want + 1e-6) for v in grads]
    half = torch.finfo(t).eps / 2

    def close(got):
        for o, r in zip(got, refs):
            assert bool(((o.double() - r).abs() <= (2 * NORM + half) * r.abs()).all())

    assert abs(float(moe.grad_norm(grads)) - want) <= NORM * want
    out = [torch.full_like(v, 3.0) for v in grads]           # of the same strides
    assert abs(float(moe.clip_grads(grads, 1.0, out=out)) - want) <= NORM * want
    close(out)
    moe.clip_grads(grads, 1.0)
    close(grads)


def test_a_transposed_parameter():
    moe = lib()
    w = torch.nn.Parameter(torch.randn((64, 32), generator=torch.Generator().manual_seed(1)).to(dev()).t())
    b = torch.nn.Parameter(torch.zeros(64, device=dev()))
    x = torch.randn((10, 64), generator=torch.Generator().manual_seed(2)).to(dev())
    ((x + b) @ w.t()).square().sum().backward()
    assert not w.grad.is_contiguous()
    before = w.grad.double()
    want = float((before.square().sum() + b.grad.double().square().sum()).sqrt())
    norm = moe.clip_grad_norm([w, b], 0.5 * want)
    assert abs(float(norm) - want) <= NORM * want
    assert bool(((w.grad.double() - 0.5 * before).abs() <= (2 * NORM + 2.0 ** -24) * before.abs()).all())


def test_layouts_that_are_refused():
    """Gaps, overlaps, and an out whose elements lie elsewhere."""
    moe = lib()
    a = torch.ones((6, 8), device=dev())
    for grads, out in (([a[:, :4]], None), ([a[::2]], None), ([a[:1].expand(6, 8)], None), ([a.t()], [torch.ones((8, 6), device=dev())]),
                       ([a], [torch.ones((8, 6), device=dev()).t()]), ([a.t()], [torch.ones(48, device=dev())]),
                       ([a[:, :4].contiguous()], [a[:, :4]])):
        with pytest.raises(ValueError):
            moe.clip_grads(grads, 1.0, out=out)
    assert bool((a == 1).all())
