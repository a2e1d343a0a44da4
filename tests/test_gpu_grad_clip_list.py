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
