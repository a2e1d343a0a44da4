"""The norm over a list of gradients, and their clipping, against 64 bits.

Tolerances: a thread's sum of 64 squares in fp32 is off by at most 65 u of
itself (u = 2^-24; every term is positive), so the norm by 33 u, and 1 u for
its rounding: 2^-18 is more.  The scale adds 3 u, an output half a step of
its type."""
import math

import pytest
import torch

from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -18


def tensors(sizes, seed=0, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device=dev())).to(t) for n, t in sizes]


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(moe, grads, max_norm, inplace=False, eps=1e-6):
    want = norm64(grads)
    scale = min(1.0, max_norm / (want + eps))
    refs = [scale * g.double() for g in grads]
    out = grads if inplace else [torch.full_like(g, 7.0) for g in grads]
    alone = moe.grad_norm(grads)
    norm = moe.clip_grads(grads, max_norm, eps=eps) if inplace else moe.clip_grads(grads, max_norm, out=out, eps=eps)
    assert norm.shape == () and norm.dtype == torch.float32 and torch.equal(norm, alone)
    if want > torch.finfo(torch.float32).max:   # rounded to fp32
        assert float(norm) == math.inf
    else:
        assert abs(float(norm) - want) <= NORM * want
    for o, r in zip(out, refs):
        half = torch.finfo(o.dtype).eps / 2
        least = torch.finfo(o.dtype).smallest_normal * half * 2   # half a step below the normal range
        assert bool(((o.double() - r).abs() <= (2 * NORM + half) * r.abs() + least).all())


F, B = torch.float32, torch.bfloat16
LISTS = {"one": [(1, F)], "one bf16": [(1, B)], "odd": [(1001, F), (7, B), (3, F), (16385, B), (1, B)],
         "chunks": [(16384, F), (16384, B), (32768, B), (16383, F), (16385, F)], "empty among": [(0, F), (5, B), (0, B), (9, F)],
         "only empty": [(0, F), (0, B)], "large": [(5000001, F), (3000001, B)], "many": [(17 * i % 300 + 1, F if i % 3 else B) for i in range(700)],
         "limits": [(100, F)] * 512, "and one more": [(100, B)] * 513}


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("max_norm", (0.5, 1e9))
@pytest.mark.parametrize("inplace", (False, True))
def test_lists(name, max_norm, inplace):
    check(lib(), tensors(LISTS[name]), max_norm, inplace)


@pytest.mark.parametrize("offset", range(9))
@pytest.mark.parametrize("t", (F, B))
def test_alignment(offset, t):
    """Views at every offset of their type, into buffers of the same and of another offset."""
    moe = lib()
    flat = tensors([(40000, t)])[0]
    grads = [flat[offset:offset + 17000], flat[20000 + offset:20000 + 2 * offset + 1]]
    want = norm64(grads)
    scale = 1.0 / (want + 1e-6)
    for shift in (0, 1, 4):
        buffer = torch.full((20000,), 3.0, dtype=t, device=dev())
        at = offset + shift
        out = [buffer[at:at + 17000], buffer[at + 17000:at + 17000 + grads[1].numel()]]
        norm = moe.clip_grads(grads, 1.0, out=out)
        assert abs(float(norm) - want) <= NORM * want
        for o, g in zip(out, grads):
            assert bool(((o.double() - scale * g.double()).abs() <= (2 * NORM + torch.finfo(t).eps / 2) * scale * g.double().abs() + 1e-40).all())
        assert bool((buffer[:at] == 3).all()) and bool((buffer[at + 17000 + grads[1].numel():] == 3).all())


@pytest.mark.parametrize("t,scale", ((F, 1e-30), (F, 1e-38), (F, 1e-42), (F, 1e25), (F, 1e37), (B, 1e-30), (B, 1e30), (B, 1e-39), (F, 2.0 ** -41), (F, 2.0 ** 62)))
def test_values_whose_squares_fp32_does_not_hold(t, scale):
    moe = lib()
    grads = tensors([(1000, t), (20000, t), (33, t)], scale=1.0)
    grads = [(g.double() * scale).to(t) for g in grads]
    assert any(float(g.abs().max()) > 0 for g in grads)
    check(moe, grads, 1.0)
    mixed = grads + tensors([(500, F)])     # with ordinary ones
    check(moe, mixed, 1.0)


def test_zeros_infinities_and_nan():
    """As the formula says: zeros stay, an infinity gives a scale of 0 (itself NaN), NaN spreads."""
    moe = lib()
    grads = [torch.zeros(50000, device=dev()), torch.zeros(77, dtype=B, device=dev())]
    assert float(moe.clip_grads(grads, 1.0)) == 0 and all(bool((g == 0).all()) for g in grads)
    grads = tensors([(20000, F), (100, B)])
    grads[0][12345] = float("inf")
    assert float(moe.grad_norm(grads)) == math.inf
    moe.clip_grads(grads, 1.0)
    assert bool(grads[0][12345].isnan()) and float(grads[0][:12345].abs().max()) == 0 and float(grads[1].abs().max()) == 0
    grads = tensors([(20000, F), (100, B)])
    grads[1][3] = float("nan")
    assert math.isnan(float(moe.clip_grads(grads, 1.0))) and all(bool(g.isnan().all()) for g in grads)
    huge = [torch.full((100,), 3e38, device=dev())]      # finite values, a norm beyond fp32
    assert float(moe.grad_norm(huge)) == math.inf


def test_shapes_and_parameters():
    """Tensors of any shape, and a max_norm of 0 or infinity."""
    moe = lib()
    grads = [t.view(s) for t, s in zip(tensors([(12, F), (30, B), (1, F)]), ((3, 4), (5, 2, 3), ()))]
    want = norm64(grads)
    assert abs(float(moe.clip_grads(tuple(grads), math.inf)) - want) <= NORM * want
    moe.clip_grads(grads, 0.0)
    assert all(bool((g == 0).all()) for g in grads)


def test_more_than_32_bits_of_elements():
    """A tensor of 2^32 + 5 elements, as large layers have."""
    moe = lib()
    n = 2 ** 32 + 5
    g = torch.zeros(n, dtype=B, device=dev())
    g[0], g[2 ** 31 + 1], g[2 ** 32 + 4] = 3.0, 4.0, 12.0
    assert float(moe.clip_grads([g], 6.5)) == 13.0
    assert g[0] == 1.5 and g[2 ** 31 + 1] == 2.0 and g[2 ** 32 + 4] == 6.0


def test_the_same_every_time_in_a_graph_and_on_another_stream():
    moe = lib()
    grads = tensors([(300000, F), (12345, B), (1, F)])
    out = [torch.empty_like(g) for g in grads]
    want = moe.clip_grads(grads, 1.0, out=out)
    kept = [o.clone() for o in out]
    for _ in range(5):
        assert torch.equal(moe.clip_grads(grads, 1.0, out=out), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = moe.clip_grads(grads, 1.0, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want) and all(torch.equal(a, b) for a, b in zip(out, kept))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = moe.clip_grads(grads, 1.0, out=out)
    for g in grads:
        g *= 2
    for o in out:
        o.zero_()
    graph.replay()
    assert torch.equal(norm, moe.grad_norm(grads))
    assert abs(norm64(out) - 1.0) < 1e-3


def test_refusals():
    moe = lib()
    a, b = tensors([(64, F), (64, F)])
    flat = torch.zeros(100, device=dev())
    for grads, out in (([], None), ([a, a], None), ([flat[:60], flat[50:]], None), ([a, b], [a]), ([a, b], [a, a]), ([a, b], [b, a]),
                       ([a], [flat[:60]]), ([a], [a.to(B)]), ([a.half()], None), ([a.cpu()], None), ([a[::2]], None), (a, None),
                       ([a], [flat[::2][:64]]), ([None], None), ([a, flat[:30]], [flat[:64], flat[70:100]])):
        with pytest.raises((ValueError, TypeError)):
            moe.clip_grads(grads, 1.0, out=out)
    for max_norm, eps in ((-1.0, 1e-6), (math.nan, 1e-6), (1.0, -1.0), (1.0, math.nan)):
        with pytest.raises(moe.MoEError):
            moe.clip_grads([a], max_norm, eps=eps)
    assert abs(float(moe.grad_norm([a, a])) - math.sqrt(2) * norm64([a])) <= NORM * 2 * norm64([a])   # read only: any overlap
