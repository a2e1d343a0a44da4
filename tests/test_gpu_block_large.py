"""Offsets beyond 32 bits in the few-token experts and the norms around a
block, and choices whose masked logits hold the type's lowest value."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_few import close, reference, weights

pytestmark = pytest.mark.gpu


def test_the_last_experts_of_large_weights():
    """64 experts of H 7168, I 2560: 2.3 G weights, of which the last two are used."""
    moe = lib()
    T, H, E, k, I = 5, 7168, 64, 2, 2560
    gate_up = torch.zeros((E * H, 2 * I), dtype=torch.bfloat16, device=dev())
    down = torch.zeros((E * I, H), dtype=torch.bfloat16, device=dev())
    gate_up[-2 * H:], down[-2 * I:] = weights(2, H, I, 3)
    g = torch.Generator(device=dev()).manual_seed(4)
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    ids = torch.tensor([[63, 62]] * T, dtype=torch.int32, device=dev())
    w = torch.rand((T, k), generator=g, device=dev())
    y = moe.experts_few(x, ids, w, gate_up, down)
    moe.sync_status()
    close(y, reference(x, ids - 62, w, gate_up[-2 * H:], down[-2 * I:]))


@pytest.mark.parametrize("gates", (1, 270000))
def test_rows_beyond_2_31_elements(gates):
    """270000 rows of 8192: the last rows forward and backward are those of a call on them alone."""
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
    r, h, stats = moe.block_norm(x, weight, branch, gate=gate, save_for_backward=True)
    grads = moe.block_norm_bwd(dh, dr, x, stats, weight, branch, gate=gate)
    kw = dict(gate=gate[-min(tail, gates):].contiguous())
    rows = [t[-tail:].contiguous() for t in (x, branch, dh, dr)]
    r2, h2, stats2 = moe.block_norm(rows[0], weight, rows[1], save_for_backward=True, **kw)
    some = moe.block_norm_bwd(rows[2], rows[3], rows[0], stats2, weight, rows[1], **kw)
    moe.sync_status()
    assert torch.equal(r[-tail:], r2) and torch.equal(h[-tail:], h2)
    assert torch.equal(grads["dx"][-tail:], some["dx"]) and torch.equal(grads["d_branch"][-tail:], some["d_branch"])
    assert bool((r[:-tail] == 0).all()) and bool((grads["dx"][:-tail] == 0).all())
    # the other rows add zeros to the sums
    for n in ("d_weight", "d_gate"):
        a, b = grads[n][-tail:] if n == "d_gate" and gates > 1 else grads[n], some[n]
        half = torch.finfo(a.dtype).eps / 2
        scale = sum((rows[2].float().abs() * rows[i].float().abs()).sum(0).max() for i in (0, 1)) * 8 + dr.abs().max() * 16
        assert float((a.double() - b.double()).abs().max()) <= float(scale) * (2.0 ** -18 + (half if a.dtype == torch.bfloat16 else 0))


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_logits_masked_by_the_lowest_value(score):
    """A mask of fp32's lowest value instead of -inf: those experts come last, with weight 0."""
    moe = lib()
    T, H, E, k, I = 4, 128, 8, 6, 64
    gu, dn = weights(E, H, I, 5)
    g = torch.Generator(device=dev()).manual_seed(6)
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    wr = torch.randn((H, E), generator=g, device=dev()) / 16
    bias = torch.zeros(E, device=dev())
    bias[[1, 4, 6]] = torch.finfo(torch.float32).min
    y, ids, w = moe.layer_few(x, wr, gu, dn, k, bias=bias, score=score)
    moe.sync_status()
    assert set(ids[:, :5].reshape(-1).tolist()) == {0, 2, 3, 5, 7} and bool((w[:, 5:] == 0).all()) and bool(w.isfinite().all())
    assert bool(((w.double().sum(1) - 1).abs() <= 2.0 ** -20).all())
    close(y, reference(x, ids, w, gu, dn))
    bias.fill_(torch.finfo(torch.float32).min)        # all of them: still finite
    y, ids, w = moe.layer_few(x, wr, gu, dn, k, bias=bias, score=score)
    assert bool(w.isfinite().all()) and bool(y.isfinite().all())
