"""The norms around a block where rows are wide: dr outside the ring, vectors
outside the shared memory, rows' own gates; and operands that hold zeros.
Tolerances as in test_gpu_block_norm."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_block_norm import inputs, run_both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", (3952, 4104, 7168, 7904, 8192))
@pytest.mark.parametrize("x,gate", (("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")))
@pytest.mark.parametrize("post", (None, "bf16", "f32"))
@pytest.mark.parametrize("T,gates", ((306, 0), (306, 1), (306, 6), (306, 153), (306, 306)))
def test_wide_rows(H, x, gate, post, T, gates):
    if gates == 0 and gate == "bf16":
        pytest.skip("no gate")
    d, up = inputs(T, H, x=x, post=post, gates=gates, gate=gate)
    run_both(lib(), d, up, 0.7, 0.5)


@pytest.mark.parametrize("weight", (None, "f32"))
@pytest.mark.parametrize("gates", (1, 4, 400))
@pytest.mark.parametrize("post", (None, "f32"))
def test_zeros(weight, gates, post):
    """A gate of zero has a gradient, and so has a norm's weight of zero; each takes the other's."""
    d, up = inputs(400, 520, weight=weight, post=post, gates=gates)
    d["gate"][:, ::3] = 0
    if post:
        d["post_weight"][1::3] = 0
        d["post_weight"][3::6] = 0
    d["branch"][7] = 0
    _, _, _, grads = run_both(lib(), d, up)
    assert bool((grads["d_gate"][:, ::6] != 0).any())
    if post:
        assert bool((grads["d_post_weight"][::3] == 0).all()) and bool((grads["d_gate"][:, 1::3] == 0).all())
        assert bool((grads["d_post_weight"][1::3] != 0).any())


@pytest.mark.parametrize("gates", (2, 8, 64))
def test_the_same_bits_again(gates):
    """Sums over ranges and groups have a fixed order."""
    moe = lib()
    d, up = inputs(8192, 1024, post="f32", gates=gates)
    a = run_both(moe, d, up)[3]
    for _ in range(3):
        b = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], moe.block_norm(d["x"], d["weight"], d["branch"], post_weight=d["post_weight"],
                               gate=d["gate"], save_for_backward=True)[2], d["weight"], d["branch"], post_weight=d["post_weight"], gate=d["gate"])
        assert all(torch.equal(a[n], b[n]) for n in a)
