"""The sigmoid's scores for every fp32 logit."""
import pytest
import torch

from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu


def test_every_logit():
    """1 / (1 + exp(-z)), each step rounded to fp32, bit for bit, for all 2^32
    bit patterns of z (NaN for NaN): the weights of a choice of all 32 of a
    row's experts, neither renormalised nor scaled."""
    moe = lib()
    E = 32
    step = 1 << 27
    for first in range(-2 ** 31, 2 ** 31, step):
        z = torch.arange(first, first + step, dtype=torch.int64, device=dev()).to(torch.int32).view(torch.float32).view(-1, E)
        want = 1 / (1 + torch.exp(-z))
        ids, w = moe.route_select(z, E, score="sigmoid", renorm=False)
        want = want.gather(1, ids.long())
        assert bool(((w.view(torch.int32) == want.view(torch.int32)) | (w.isnan() & want.isnan())).all()), hex(first)
        del z, want, ids, w
    moe.sync_status()


def test_every_logit_by_its_score():
    """The same scores where they choose: with a bias of zeros the order of a
    row is that of the rounded scores, equal ones by their index."""
    moe = lib()
    E = 32
    zero = torch.zeros(E, device=dev())
    step = 1 << 24
    g = torch.Generator(device=dev()).manual_seed(3)
    for first in range(0, 2 ** 32, 1 << 28):
        z = (first + torch.randint(0, 1 << 28, (step,), generator=g, device=dev())).to(torch.int32).view(torch.float32).view(-1, E)
        z = torch.where(z.isnan(), 0.0, z)
        s = 1 / (1 + torch.exp(-z))
        value = torch.where(z == float("-inf"), float("-inf"), s)
        ids, w = moe.route_select(z, E, bias=zero, score="sigmoid", renorm=False)
        want = torch.sort(value, dim=1, descending=True, stable=True).indices
        assert torch.equal(ids.long(), want) and torch.equal(w, s.gather(1, want)), hex(first)
    moe.sync_status()
