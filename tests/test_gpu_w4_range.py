"""The 4-bit experts where single values of a row are far above the others,
or infinite, against the 64-bit references and their bounds (test_gpu_w4):
the kernel of few slots, and the other one.
"""
import numpy as np
import pytest
import torch

import ref_select as ref
from gpu_helpers import dev, f64, i32, lib
from test_gpu_w4 import check_down, check_gate_up, dev_of, ids_of, rows_of, weights

pytestmark = pytest.mark.gpu

E, K_TOKEN = 5, 2
TOKENS = {"few slots": 2, "many slots": 100}


def sizes(kernel, columns):
    """T of a call that takes the kernel: few slots run where all their blocks fit
    on the GPU at once, two on each of its multiprocessors."""
    T = TOKENS[kernel]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (columns // 64 * T * K_TOKEN <= 2 * sms) if kernel == "few slots" else (columns // 64 * T > 2 * sms)
    return T


def codes_at(q, k, zero):
    """Words q with the codes of row k set to zero ([N], or one value), for every expert."""
    K = q.shape[0] * 8 // E
    words = q.view(np.uint32).reshape(E, K // 8, -1).copy()
    shift = np.uint32(4 * (k % 8))
    words[:, k // 8] &= ~(np.uint32(15) << shift)
    words[:, k // 8] |= zero.astype(np.uint32) << shift
    return words.reshape(q.shape).view(np.int32)


def on_the_zeros(q, scales, z, group, ks):
    """The codes of rows ks equal to their zeros: terms of 0 whatever the row holds there."""
    rows = scales.shape[0] // E
    for k in ks:
        zero = np.full((E, scales.shape[1]), 8) if z is None else z.reshape(E, rows, -1)[:, k // group]
        q = codes_at(q, k, zero)
    return q, scales, z


def spiked(rows, ks, value):
    """Small rows (0.01) but for `value` at ks, its sign alternating."""
    rows = (0.01 * rows.float()).bfloat16()
    for i, k in enumerate(ks):
        rows[..., k] = value * (-1) ** i
    return rows


@pytest.mark.parametrize("kernel", TOKENS)
@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("zeros", (False, True))
@pytest.mark.parametrize("spike", (2.0 ** 14, 2.0 ** 40))
def test_large_values_on_codes_equal_to_their_zero(kernel, group, zeros, spike):
    """scale * (q - zero) x is 0 there, however large x: the result is that of
    the other terms, within the bound on the terms' own magnitudes."""
    moe = lib()
    K, N = 512, 512
    T = sizes(kernel, N)
    ks = [0, 37, 130, 255, 256, 511]
    ids = ids_of(1, T, E, K_TOKEN)
    up = on_the_zeros(*weights(group, E, K, N, group, zeros), group, ks)
    check_gate_up(moe, spiked(rows_of(3, T, K), ks, spike), ids, *up, group)
    down = on_the_zeros(*weights(group + 1, E, K, N, group, zeros), group, ks)
    w = np.random.default_rng(2).normal(size=(T, K_TOKEN)).astype(np.float32)
    check_down(moe, spiked(rows_of(4, T, K_TOKEN, K), ks, spike), ids, w, *down, group)


@pytest.mark.parametrize("kernel", TOKENS)
def test_rows_whose_mean_is_not_zero(kernel):
    """Rows of 1 + a little on codes near their zero."""
    moe = lib()
    K, N, group = 1024, 512, 128
    T = sizes(kernel, N)
    q, scales, _ = weights(1, E, K, N, group, False)
    codes = np.random.default_rng(7).integers(7, 10, size=(q.shape[0], 8, N)).astype(np.uint32)
    q = sum(codes[:, i] << np.uint32(4 * i) for i in range(8)).view(np.int32)
    ids = ids_of(1, T, E, K_TOKEN)
    rows = (1 + 0.01 * rows_of(3, T, K_TOKEN, K).float()).bfloat16()
    check_gate_up(moe, rows[:, 0].contiguous(), ids, q, scales, None, group)
    check_down(moe, rows, ids, np.ones((T, K_TOKEN), np.float32), q, scales, None, group)


@pytest.mark.parametrize("kernel", TOKENS)
@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("zeros", (False, True))
def test_infinite_values(kernel, group, zeros):
    """An infinite entry: plus or minus infinity where the code is above or
    below its zero, NaN where it equals it; the other tokens as without it."""
    moe = lib()
    K, N = 256, 512
    T = sizes(kernel, N)
    ids = ids_of(1, T, E, K_TOKEN)
    for seed, value in ((1, np.inf), (2, -np.inf)):
        q, scales, z = weights(seed, E, K, N, group, zeros)
        W = ref.unpack(q, scales.float().numpy(), z, K, N, group)
        qd = dev_of(q, scales, z)
        x, h = rows_of(seed, T, K), rows_of(seed + 2, T, K_TOKEN, K)
        clean_h, clean_y = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *qd), moe.w4_down_combine(h.to(dev()), i32(ids), None, *qd)
        t, k = T // 2, 93
        x[t, k] = value
        h[t, 1, k] = value
        with np.errstate(all="ignore"):
            gu = value * W[ids[t], k]                       # [slots, N], NaN where the code equals its zero
            want_h = ref.silu(gu[:, :N // 2]) * gu[:, N // 2:]
            want_y = value * W[ids[t, 1], k]
        got_h, got_y = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *qd), moe.w4_down_combine(h.to(dev()), i32(ids), None, *qd)
        moe.sync_status()
        np.testing.assert_array_equal(f64(got_y[t]), want_y)
        assert np.isfinite(want_y).sum() == 0 and np.isinf(want_y).sum() > 0 and np.isnan(want_y).sum() > 0
        finite = np.isfinite(want_h)                        # silu(-inf) u is NaN, none is finite
        assert not finite.any()
        np.testing.assert_array_equal(f64(got_h[t]), want_h)
        keep = [i for i in range(T) if i != t]
        assert torch.equal(got_h[keep], clean_h[keep]) and torch.equal(got_y[keep], clean_y[keep])
