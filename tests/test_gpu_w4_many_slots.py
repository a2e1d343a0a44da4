"""Isolation, errors, offsets and streams of the 4-bit experts' kernel of many
slots, with its sort of up to 32 slots (8 tokens) and of more (96 tokens).

The kernel of few slots runs where its blocks all fit on the GPU at once, two a
multiprocessor: a block for every 64 columns and every slot (gate_up) or token
(down), at the least.  Each call here has more.
"""
import ctypes

import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32, i32, lib, npi
from test_gpu_w4 import check_down, check_gate_up, dev_of, ids_of, rows_of, weights

pytestmark = pytest.mark.gpu

E, K_TOKEN, GROUP = 5, 4, 64
H, I = 2816, 448
TOKENS = (8, 96)


def many(columns, slots_or_tokens):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert columns // 64 * slots_or_tokens > 2 * sms


def calls_are_of_many(T):
    many(2 * I, T * K_TOKEN)
    many(H, T)


@pytest.fixture(scope="module")
def experts():
    return weights(1, E, H, 2 * I, GROUP, False), weights(2, E, I, H, GROUP, True)


def some_empty(T):
    """Every expert more than once, empty slots and two padded tokens."""
    ids = ids_of(3, T, E, K_TOKEN)
    ids[[2, T - 1]] = -1
    ids[5, 0] = ids[4, 3] = -1
    return ids


@pytest.mark.parametrize("T", TOKENS)
def test_nothing_leaks_from_empty_slots(T, experts):
    """NaN and infinities in a padded token's row, its slots' rows of h and
    their weights reach no other row; the padded rows are zero, or y_shared."""
    moe = lib()
    calls_are_of_many(T)
    qg, qd = experts
    ids = some_empty(T)
    x, h, shared = rows_of(1, T, H), rows_of(2, T, K_TOKEN, I), rows_of(4, T, H)
    w = np.random.default_rng(1).normal(size=(T, K_TOKEN)).astype(np.float32)
    clean_h, clean_y = check_gate_up(moe, x, ids, *qg, GROUP), check_down(moe, h, ids, w, *qd, GROUP)
    with_shared = check_down(moe, h, ids, w, *qd, GROUP, shared)
    x[[2, T - 1]] = float("nan")
    h[2], h[T - 1], h[5, 0], h[4, 3] = float("inf"), float("nan"), float("nan"), float("-inf")
    w[[2, T - 1]] = np.nan
    w[5, 0], w[4, 3] = np.inf, np.nan
    a = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(*qg))
    b = moe.w4_down_combine(h.to(dev()), i32(ids), f32(w), *dev_of(*qd))
    assert torch.equal(a, clean_h) and torch.equal(b, clean_y)
    assert float(b[[2, T - 1]].float().abs().max()) == 0
    b = moe.w4_down_combine(h.to(dev()), i32(ids), f32(w), *dev_of(*qd), y_shared=shared.to(dev()))
    assert torch.equal(b, with_shared) and torch.equal(b[[2, T - 1]].cpu(), shared[[2, T - 1]])
    nothing = torch.full((T, K_TOKEN), -1, dtype=torch.int32, device=dev())
    assert float(moe.w4_gate_up_swiglu(x.to(dev()), nothing, *dev_of(*qg)).float().abs().max()) == 0
    assert float(moe.w4_down_combine(h.to(dev()), nothing, f32(w), *dev_of(*qd)).float().abs().max()) == 0
    moe.sync_status()


@pytest.mark.parametrize("T", TOKENS)
def test_what_the_workspace_held_is_not_used(T, experts):
    """The products of empty slots are never written: NaN left there by an
    earlier user of the memory stay out of y."""
    moe = lib()
    many(H, T)
    qd = experts[1]
    ids = some_empty(T)
    h = rows_of(2, T, K_TOKEN, I)
    w = np.random.default_rng(1).normal(size=(T, K_TOKEN)).astype(np.float32)
    want = check_down(moe, h, ids, w, *qd, GROUP)
    size = ctypes.c_size_t(0)
    moe._lib.call("moe_w4_down_workspace_size", T, H, K_TOKEN, ctypes.byref(size))
    ws = torch.full((size.value // 4,), float("nan"), device=dev())
    y = torch.empty_like(want)
    hd, idd, wd, (q, s, z) = h.to(dev()), i32(ids), f32(w), dev_of(*qd)
    moe._lib.call("moe_w4_down_combine", hd.data_ptr(), idd.data_ptr(), wd.data_ptr(), q.data_ptr(), s.data_ptr(), z.data_ptr(),
                  None, T, H, E, K_TOKEN, I, GROUP, y.data_ptr(), ws.data_ptr(), size.value,
                  torch.cuda.current_stream().cuda_stream)
    moe.sync_status()
    assert torch.equal(y, want) and bool(ws.view(T, K_TOKEN, H)[2].isnan().all())


@pytest.mark.parametrize("T", TOKENS)
def test_a_nan_row_stays_in_its_row(T, experts):
    """The other rows of its expert, of the same products of matrices, keep their bits."""
    moe = lib()
    calls_are_of_many(T)
    qg, qd = experts
    ids = ids_of(3, T, E, K_TOKEN)
    x, h = rows_of(1, T, H), rows_of(2, T, K_TOKEN, I)
    clean_h = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(*qg))
    clean_y = moe.w4_down_combine(h.to(dev()), i32(ids), None, *dev_of(*qd))
    assert (np.bincount(ids.ravel(), minlength=E) > 1).all()
    x[4, 100] = float("nan")
    h[4, 1, 60] = float("nan")
    a = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(*qg))
    b = moe.w4_down_combine(h.to(dev()), i32(ids), None, *dev_of(*qd))
    keep = [t for t in range(T) if t != 4]
    assert torch.equal(a[keep], clean_h[keep]) and bool(a[4].isnan().all())
    assert torch.equal(b[keep], clean_y[keep]) and bool(b[4].isnan().all())
    moe.sync_status()


@pytest.mark.parametrize("T", TOKENS)
def test_bad_ids_are_reported(T, experts):
    """An id outside [0, E) but -1: MOE_ERR_DEVICE, an empty slot, and the other
    tokens' bits; from gate_up, and from down with its combine."""
    moe = lib()
    calls_are_of_many(T)
    qg, qd = (dev_of(*q) for q in experts)
    x = rows_of(1, T, H).to(dev())
    ids = i32(ids_of(3, T, E, K_TOKEN))
    good = moe.w4_gate_up_swiglu(x, ids, *qg)
    empty = ids.clone()
    empty[1, 1] = -1
    want_h, want_y = moe.w4_gate_up_swiglu(x, empty, *qg), moe.w4_down_combine(good, empty, None, *qd)
    moe.sync_status()
    for bad in (E, -2, 2 ** 31 - 1, -2 ** 31):
        wrong = ids.clone()
        wrong[1, 1] = bad
        for call, want in ((lambda: moe.w4_gate_up_swiglu(x, wrong, *qg), want_h),
                           (lambda: moe.w4_down_combine(good, wrong, None, *qd), want_y)):
            got = call()
            with pytest.raises(moe.MoEError) as err:
                moe.sync_status()
            assert err.value.status == 6
            assert torch.equal(got, want)
    moe.sync_status()


@pytest.mark.parametrize("T", TOKENS)
def test_dense_expert(T):
    """ids None: one expert for every token."""
    moe = lib()
    Id, Hd = 1600, 3200   # 50 column blocks of each product
    many(2 * Id, T)
    many(Hd, T)
    qg, qd = weights(1, 1, 128, 2 * Id, GROUP, True), weights(2, 1, 128, Hd, GROUP, False)
    x, zero = rows_of(1, T, 128), np.zeros((T, 1), np.int32)
    h = moe.w4_gate_up_swiglu(x.to(dev()), None, *dev_of(*qg))
    assert torch.equal(h, check_gate_up(moe, x, zero, *qg, GROUP))
    y = moe.w4_down_combine(x.view(T, 1, 128).to(dev()), None, None, *dev_of(*qd))
    assert torch.equal(y, check_down(moe, x.view(T, 1, 128), zero, np.ones((T, 1), np.float32), *qd, GROUP))


@pytest.mark.parametrize("T", TOKENS)
def test_offsets_past_32_bits(T):
    """Experts whose words lie past 2^31 words and 2^33 bytes."""
    moe = lib()
    E_, K, N, group = 600, 7168, 4096, 128
    many(N, T)
    q = torch.empty((E_ * K // 8, N), dtype=torch.int32, device=dev())
    scales = torch.empty((E_ * K // group, N), dtype=torch.bfloat16, device=dev())
    assert q.numel() > 2 ** 31
    last = E_ - 1
    q1, s1, _ = weights(4, 1, K, N, group, False)
    q[last * K // 8:] = torch.from_numpy(q1).to(dev())
    scales[last * K // group:] = s1.to(dev())
    x = rows_of(1, T, K).to(dev())
    at = torch.full((T, 1), last, dtype=torch.int32, device=dev())
    zero = torch.zeros((T, 1), dtype=torch.int32, device=dev())
    one = dev_of(q1, s1, None)
    assert torch.equal(moe.w4_gate_up_swiglu(x, at, q, scales), moe.w4_gate_up_swiglu(x, zero, *one))
    assert torch.equal(moe.w4_down_combine(x.view(T, 1, K), at, None, q, scales),
                       moe.w4_down_combine(x.view(T, 1, K), zero, None, *one))
    moe.sync_status()


@pytest.mark.parametrize("T", TOKENS)
def test_another_stream(T, experts):
    """The product and its combine behind the work that writes their rows, on a stream of their own."""
    moe = lib()
    calls_are_of_many(T)
    qg, qd = (dev_of(*q) for q in experts)
    ids = i32(some_empty(T))
    x, w = rows_of(1, T, H).to(dev()), f32(np.random.default_rng(1).random((T, K_TOKEN)))
    h0 = moe.w4_gate_up_swiglu(x + x, ids, *qg)
    y0 = moe.w4_down_combine(h0, ids, w, *qd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=dev())
        for _ in range(4):
            big = big @ big * 1e-3
        h = moe.w4_gate_up_swiglu(x + x, ids, *qg)
        y = moe.w4_down_combine(h, ids, w, *qd)
    s.synchronize()
    assert torch.equal(h, h0) and torch.equal(y, y0)
    moe.sync_status()


@pytest.mark.parametrize("T", TOKENS)
def test_the_same_call_gives_the_same_bits(T, experts):
    """Twenty times, with other calls in between."""
    moe = lib()
    calls_are_of_many(T)
    qg, qd = (dev_of(*q) for q in experts)
    ids = i32(some_empty(T))
    other = i32(np.ascontiguousarray(npi(ids)[::-1]))
    x, w = rows_of(1, T, H).to(dev()), f32(np.random.default_rng(1).random((T, K_TOKEN)))
    h = moe.w4_gate_up_swiglu(x, ids, *qg)
    y = moe.w4_down_combine(h, ids, w, *qd)
    for _ in range(20):
        moe.w4_down_combine(moe.w4_gate_up_swiglu(x, other, *qg), other, w, *qd)
        assert torch.equal(moe.w4_gate_up_swiglu(x, ids, *qg), h) and torch.equal(moe.w4_down_combine(h, ids, w, *qd), y)
    moe.sync_status()
