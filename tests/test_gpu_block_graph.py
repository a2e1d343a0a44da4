"""A training step of a block, with clipped gradients, captured into a CUDA
graph and replayed on new inputs: an eager step's bits."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_block import H, make, stream

pytestmark = pytest.mark.gpu


def step(moe, block, x, dr):
    r, _ = block(x)
    r.backward(dr)
    return r, moe.clip_grad_norm(block.parameters(), 1.0)


@pytest.mark.parametrize("routed", (False, True))
def test_a_captured_training_step(routed):
    moe = lib()
    routing = moe.Routing(score="sigmoid", n_groups=4, top_groups=2, scale=2.5) if routed else None
    kw = dict(post_norm=True, learned_scale=0.5, routing=routing)
    block, eager = make(moe, 3, **kw), make(moe, 3, **kw)
    x, dr = stream(64, torch.float32), stream(64, torch.float32, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # one-time set-up outside the capture
        for _ in range(2):
            block.zero_grad(set_to_none=True)
            step(moe, block, x, dr)
    torch.cuda.current_stream().wait_stream(side)
    block.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, norm = step(moe, block, x, dr)
    for seed in (1, 7, 8):
        x.copy_(stream(64, torch.float32, seed))
        dr.copy_(stream(64, torch.float32, seed + 20))
        graph.replay()
        eager.zero_grad(set_to_none=True)
        want, want_norm = step(moe, eager, x, dr)
        assert torch.equal(r, want) and torch.equal(norm, want_norm)
        for p, q in zip(block.parameters(), eager.parameters()):
            assert torch.equal(p.grad, q.grad)
    moe.sync_status()


def test_no_tokens():
    """An empty batch through a block: gradients of zeros, a norm of 0."""
    moe = lib()
    block = make(moe, post_norm=True, learned_scale=0.5)
    x = torch.zeros((0, H), device=dev(), requires_grad=True)
    r, h = block(x, next_norm=torch.ones(H, device=dev()))
    assert r.shape == h.shape == (0, H)
    (r.sum() + h.float().sum()).backward()
    assert x.grad.shape == (0, H) and all(bool((p.grad == 0).all()) for p in block.parameters() if p.grad is not None)
    assert float(moe.clip_grad_norm(block.parameters(), 1.0)) == 0.0
    r, h = block.decode(x.detach(), next_norm=torch.ones(H, device=dev()))
    assert r.shape == h.shape == (0, H)
    moe.sync_status()
