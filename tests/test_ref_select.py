"""The 64-bit references of the expert choice: brute force, and their gradient
against central differences of their forward (CPU)."""
import itertools

import numpy as np
import pytest

import ref_select as ref


@pytest.mark.parametrize("score,renorm", itertools.product(("softmax", "sigmoid"), (True, False)))
def test_gradient_is_the_differences(score, renorm):
    """sum(w * dw) of the chosen weights moved by +-h in each logit; the error
    of a central difference is h^2/6 times a third derivative of order one,
    plus 2^-53 / h."""
    rng = np.random.default_rng(3)
    T, E, k, scale, h = 5, 12, 3, 2.5, 1e-4
    z, dw = rng.normal(size=(T, E)), rng.normal(size=(T, k))
    ids = ref.select(z, k, score=score, n_groups=3, top_groups=2, group_score="max")["ids"]
    d = ref.select_bwd(dw, z, ids, score, renorm, scale)
    for e in range(E):
        zp, zm = z.copy(), z.copy()
        zp[:, e] += h
        zm[:, e] -= h
        diff = ((ref.weights_of(zp, ids, score, renorm, scale) - ref.weights_of(zm, ids, score, renorm, scale)) * dw).sum(1) / (2 * h)
        np.testing.assert_allclose(d[:, e], diff, atol=10 * scale * h * h)


def test_choice_by_hand():
    z = np.log(np.array([[0.1, 0.2, 0.05, 0.25, 0.3, 0.1]]))
    r = ref.select(z, 2, n_groups=3, top_groups=1, group_score="top2")
    assert r["ids"].tolist() == [[4, 5]]          # 0.3, 0.3, 0.4
    r = ref.select(z, 2, n_groups=3, top_groups=2, group_score="max", scale=2.0)
    assert r["ids"].tolist() == [[4, 3]]
    np.testing.assert_allclose(r["w"], [[2 * 0.3 / 0.55, 2 * 0.25 / 0.55]])
    r = ref.select(z, 2, bias=[1.0, 0, 1.0, 0, 0, 0], renorm=False)
    assert r["ids"].tolist() == [[0, 2]]          # the bias chooses, the scores weigh
    np.testing.assert_allclose(r["w"], [[0.1, 0.05]])
