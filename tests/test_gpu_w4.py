"""The 4-bit experts on the GPU against 64-bit references.

Bounds: a sum of K exact products accumulated in fp32 is off by at most
(K + 16) * 2^-23 of the sum of the terms' magnitudes (2^-23 an addition: the
tensor cores may truncate; 16 for the group scales' products and the joins);
h = silu(g) u adds |u| * 1.1 dg + |silu(g)| du and 16 * 2^-24 |h| for the
exponential and the quotient; a bf16 result half an ulp.
"""
import numpy as np
import pytest
import torch

import ref_select as ref
from gpu_helpers import bf, dev, f32, f64, i32, lib, npi

pytestmark = pytest.mark.gpu


def weights(seed, E, K, N, group, zeros):
    g = np.random.default_rng(seed)
    q = g.integers(0, 2 ** 32, size=(E * K // 8, N), dtype=np.uint32).view(np.int32)
    scales = torch.from_numpy((g.uniform(0.5, 1.5, size=(E * K // group, N)) / (4.6 * np.sqrt(K))).astype(np.float32)).bfloat16()
    z = g.integers(0, 16, size=scales.shape).astype(np.uint8) if zeros else None
    return q, scales, z


def dev_of(q, scales, z):
    return (torch.from_numpy(q).to(dev()), scales.to(dev()), None if z is None else torch.from_numpy(z).to(dev()))


def ids_of(seed, T, E, k, empty=0.0):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[g.random((T, k)) < empty] = -1
    return ids


def rows_of(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=shape).astype(np.float32)).bfloat16()


def check_gate_up(moe, x, ids, q, scales, z, group):
    T, H = x.shape
    N = q.shape[1]
    k = ids.shape[1]
    W = ref.unpack(q, scales.float().numpy(), z, H, N, group)
    h = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(q, scales, z))
    moe.sync_status()
    assert tuple(h.shape) == (T, k, N // 2) and h.dtype == torch.bfloat16
    rows = np.repeat(x.double().numpy()[:, None], k, 1)
    gu, mag = ref.experts(rows, ids, W)
    I = N // 2
    g, u = gu[..., :I], gu[..., I:]
    dg, du = (mag[..., :I] * (H + 16) * 2.0 ** -23, mag[..., I:] * (H + 16) * 2.0 ** -23)
    want = ref.silu(g) * u
    tol = (1.1 * dg * (np.abs(u) + du) + np.abs(ref.silu(g)) * du) * 1.01 + 2.0 ** -20 * np.abs(want)
    tol = tol + ref.half_ulp_bf16(np.abs(want) + tol)
    err = np.abs(f64(h) - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert (f64(h)[ids < 0] == 0).all()
    return h


def check_down(moe, h, ids, w, q, scales, z, group, y_shared=None):
    T, k, I = h.shape
    H = q.shape[1]
    W = ref.unpack(q, scales.float().numpy(), z, I, H, group)
    y = moe.w4_down_combine(h.to(dev()), i32(ids), f32(w), *dev_of(q, scales, z),
                            y_shared=None if y_shared is None else y_shared.to(dev()))
    moe.sync_status()
    assert tuple(y.shape) == (T, H) and y.dtype == torch.bfloat16
    rows = np.where(ids[..., None] >= 0, h.double().numpy(), 0.0)
    p, mag = ref.experts(rows, ids, W)
    ww = np.where(ids >= 0, w.astype(np.float64), 0.0)[..., None]
    want = (p * ww).sum(1)
    tol = (mag * np.abs(ww)).sum(1) * (I + k + 16) * 2.0 ** -23
    if y_shared is not None:
        want = want + y_shared.double().numpy()
        tol = tol + 2.0 ** -23 * np.abs(want)
    tol = tol + ref.half_ulp_bf16(np.abs(want) + tol)
    err = np.abs(f64(y) - want)
    assert (err <= tol).all(), float((err / tol).max())
    return y


SHAPES = [  # T, H, E, k, I, group, zeros, empty
    (1, 64, 4, 2, 64, 64, False, 0.0), (1, 256, 8, 8, 128, 128, True, 0.0), (2, 192, 5, 3, 320, 32, True, 0.0),
    (3, 2048, 16, 4, 768, 128, False, 0.0), (5, 320, 3, 3, 192, 64, False, 0.3), (8, 128, 4, 1, 64, 32, False, 0.0),
    (9, 512, 4, 4, 128, 128, True, 0.2), (17, 384, 60, 6, 256, 64, True, 0.1), (33, 128, 2, 2, 448, 64, False, 0.0),
    (64, 256, 32, 8, 128, 128, False, 0.05), (70, 640, 8, 5, 64, 64, True, 0.0), (130, 64, 3, 2, 128, 32, False, 0.5),
    (300, 128, 128, 8, 64, 64, False, 0.0),
    # more than eight items for each of the GPU's blocks: whole items a warp, then shared ones; K of an odd number of
    # 64 rows, of parts of unequal length, of one part
    (64, 192, 60, 6, 1408, 64, True, 0.1), (64, 640, 60, 6, 1408, 32, False, 0.0), (40, 1152, 64, 8, 1024, 128, True, 0.0),
    (64, 2816, 60, 6, 192, 64, True, 0.1), (64, 2880, 60, 6, 640, 32, True, 0.0), (48, 4096, 64, 8, 128, 128, False, 0.0),
    # many experts: the slots of a launch row are few, so several rows
    (50, 64, 1000, 8, 64, 64, False, 0.1),
    # few slots, a warp to each part of a sum: eight parts (blocks of a cluster, one and two sums a warp), parts of
    # unequal length, the most slots a token, empty ones
    (1, 4096, 6, 4, 4160, 64, True, 0.0), (2, 64, 40, 32, 192, 32, True, 0.3), (1, 4160, 4, 2, 128, 32, False, 0.0),
    (4, 128, 9, 2, 704, 64, True, 0.4), (1, 2048, 3, 1, 2880, 64, False, 0.0), (3, 64, 33, 17, 1024, 64, False, 0.2)]


@pytest.mark.parametrize("T,H,E,k,I,group,zeros,empty", SHAPES)
def test_gate_up(T, H, E, k, I, group, zeros, empty):
    moe = lib()
    check_gate_up(moe, rows_of(T, T, H), ids_of(T + E, T, E, k, empty), *weights(H, E, H, 2 * I, group, zeros), group)


@pytest.mark.parametrize("T,H,E,k,I,group,zeros,empty", SHAPES)
def test_down(T, H, E, k, I, group, zeros, empty):
    moe = lib()
    if I % group:
        group = 64
    w = np.random.default_rng(T).normal(size=(T, k)).astype(np.float32)
    shared = rows_of(T + 3, T, H) if T % 2 else None
    check_down(moe, rows_of(T, T, k, I), ids_of(T + E, T, E, k, empty), w, *weights(H, E, I, H, group, zeros), group, shared)


def test_one_hot_rows_read_every_weight():
    """A row with one 1 gives a row of the weights exactly: scale * (q - zero)
    is a product of a 5-bit integer and a bf16, exact in fp32, rounded once."""
    moe = lib()
    E, K, N, group = 2, 256, 192, 64
    q, scales, z = weights(1, E, K, N, group, True)
    W = ref.unpack(q, scales.float().numpy(), z, K, N, group)
    qd, sd, zd = dev_of(q, scales, z)
    want = torch.from_numpy(W.astype(np.float32)).bfloat16().to(dev())
    for e in range(E):
        eye = torch.eye(K, dtype=torch.bfloat16, device=dev()).view(K, 1, K)
        y = moe.w4_down_combine(eye, torch.full((K, 1), e, dtype=torch.int32, device=dev()), None, qd, sd, zd)
        assert torch.equal(y, want[e])
    assert torch.equal(moe.w4_dequantize(qd, sd, zd), want.view(E * K, N))


def test_nothing_leaks_from_empty_slots():
    """NaN and infinities in a padded token's row, its slots' h rows and their
    weights reach no other row; the padded rows are zero (or y_shared)."""
    moe = lib()
    T, H, E, k, I, group = 12, 256, 4, 2, 128, 64
    ids = ids_of(3, T, E, k)
    ids[[2, 7, 11]] = -1
    ids[5, 0] = -1
    qg, qd = weights(1, E, H, 2 * I, group, False), weights(2, E, I, H, group, False)
    x, h = rows_of(1, T, H), rows_of(2, T, k, I)
    w = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    clean_h = check_gate_up(moe, x, ids, *qg, group)
    clean_y = check_down(moe, h, ids, w, *qd, group)
    x[[2, 7, 11]] = float("nan")
    h[[2, 11]] = float("inf")
    h[7] = float("nan")
    h[5, 0] = float("nan")
    w[[2, 7, 11]] = np.nan
    w[5, 0] = np.inf
    a = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(*qg))
    b = moe.w4_down_combine(h.to(dev()), i32(ids), f32(w), *dev_of(*qd))
    assert torch.equal(a, clean_h) and torch.equal(b, clean_y)
    assert float(b[[2, 7, 11]].float().abs().max()) == 0
    nothing = torch.full((T, k), -1, dtype=torch.int32, device=dev())
    assert float(moe.w4_gate_up_swiglu(x.to(dev()), nothing, *dev_of(*qg)).float().abs().max()) == 0
    assert float(moe.w4_down_combine(h.to(dev()), nothing, f32(w), *dev_of(*qd)).float().abs().max()) == 0
    moe.sync_status()


def test_a_nan_row_stays_in_its_row():
    moe = lib()
    T, H, E, k, I, group = 10, 128, 2, 1, 64, 64
    ids = ids_of(3, T, E, k)
    qg = weights(1, E, H, 2 * I, group, False)
    x = rows_of(1, T, H)
    clean = check_gate_up(moe, x, ids, *qg, group)
    x[4, 100] = float("nan")
    a = moe.w4_gate_up_swiglu(x.to(dev()), i32(ids), *dev_of(*qg))
    keep = [t for t in range(T) if t != 4]
    assert torch.equal(a[keep], clean[keep]) and bool(a[4].isnan().all())


def test_dense_expert():
    """ids None: one expert for every token, the shared expert's form."""
    moe = lib()
    T, H, I, group = 19, 256, 192, 64
    qg, qd = weights(1, 1, H, 2 * I, group, True), weights(2, 1, I, H, group, False)
    x = rows_of(1, T, H)
    zero = np.zeros((T, 1), np.int32)
    h = moe.w4_gate_up_swiglu(x.to(dev()), None, *dev_of(*qg))
    assert torch.equal(h, check_gate_up(moe, x, zero, *qg, group))
    y = moe.w4_down_combine(h, None, None, *dev_of(*qd))
    assert torch.equal(y, check_down(moe, h.cpu(), zero, np.ones((T, 1), np.float32), *qd, group))


@pytest.mark.parametrize("T,H,E,k,I,group", [(40, 512, 6, 3, 256, 128), (64, 2048, 64, 6, 1472, 64), (40, 4096, 16, 4, 1408, 128)])
def test_a_token_does_not_depend_on_the_batch(T, H, E, k, I, group):
    """Each token alone gives the bits it has in the batch: from the kernel of
    few slots, from items shared by a block's warps and from whole items of a
    warp."""
    moe = lib()
    ids = i32(ids_of(3, T, E, k))
    qg, qd = dev_of(*weights(1, E, H, 2 * I, group, False)), dev_of(*weights(2, E, I, H, group, False))
    x = rows_of(1, T, H).to(dev())
    w = f32(np.random.default_rng(1).random((T, k)))
    h = moe.w4_gate_up_swiglu(x, ids, *qg)
    y = moe.w4_down_combine(h, ids, w, *qd)
    for a, b in ((0, 1), (7, 9), (10, 27), (39, 40)):
        hp = moe.w4_gate_up_swiglu(x[a:b].contiguous(), ids[a:b].contiguous(), *qg)
        assert torch.equal(hp, h[a:b])
        assert torch.equal(moe.w4_down_combine(hp, ids[a:b].contiguous(), w[a:b].contiguous(), *qd), y[a:b])


def test_offsets_past_32_bits():
    """Experts whose words lie past 2^31 words and 2^33 bytes."""
    moe = lib()
    E, K, N, group = 600, 7168, 4096, 128
    q = torch.empty((E * K // 8, N), dtype=torch.int32, device=dev())
    scales = torch.empty((E * K // group, N), dtype=torch.bfloat16, device=dev())
    assert q.numel() > 2 ** 31
    last = E - 1
    q1, s1, _ = weights(4, 1, K, N, group, False)
    q[last * K // 8:] = torch.from_numpy(q1).to(dev())
    scales[last * K // group:] = s1.to(dev())
    x = rows_of(1, 3, K).to(dev())
    at = torch.full((3, 1), last, dtype=torch.int32, device=dev())
    zero = torch.zeros((3, 1), dtype=torch.int32, device=dev())
    h = moe.w4_gate_up_swiglu(x, at, q, scales)
    assert torch.equal(h, moe.w4_gate_up_swiglu(x, zero, *dev_of(q1, s1, None)))
    y = moe.w4_down_combine(x.view(3, 1, K), at, None, q, scales)
    assert torch.equal(y, moe.w4_down_combine(x.view(3, 1, K), zero, None, *dev_of(q1, s1, None)))


def test_streams_and_empty_batch():
    moe = lib()
    T, H, E, k, I, group = 32, 256, 8, 2, 128, 64
    ids = i32(ids_of(3, T, E, k))
    qg, qd = dev_of(*weights(1, E, H, 2 * I, group, False)), dev_of(*weights(2, E, I, H, group, False))
    x = rows_of(1, T, H).to(dev())
    w = f32(np.random.default_rng(1).random((T, k)))
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
    none = torch.empty((0, k), dtype=torch.int32, device=dev())
    h = moe.w4_gate_up_swiglu(x[:0], none, *qg)
    assert h.shape == (0, k, I)
    assert moe.w4_down_combine(h, none, w[:0], *qd).shape == (0, H)
    moe.sync_status()


@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("zeros", (False, True))
def test_quantize(group, zeros):
    """Scales, zeros and codes as defined, bit for bit (every step an IEEE
    fp32 operation), a group of zeros and an all-negative group; the error is
    at most half a step plus what a rounded-down scale clips."""
    moe = lib()
    rows, N = 384, 192
    g = np.random.default_rng(group)
    w = torch.from_numpy(g.normal(size=(rows, N)).astype(np.float32) * 0.1).bfloat16()
    w[:group, 0] = 0
    w[:group, 1] = -w[:group, 1].abs()
    w[:group, 2] = w[:group, 2].abs() + 1
    q, s, z = moe.w4_quantize(w.to(dev()), group, zeros=zeros)
    v = w.float().numpy().reshape(-1, group, N)
    lo, hi = np.minimum(v.min(1), np.float32(0)), np.maximum(v.max(1), np.float32(0))
    want = (hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
    sc = torch.from_numpy(want).bfloat16()
    assert torch.equal(s.cpu(), sc)
    sf = sc.float().numpy()
    safe = np.where(sf > 0, sf, np.float32(1))
    zero = np.where(sf > 0, np.minimum(np.rint(-lo / safe), 15), 0) if zeros else np.full(sf.shape, 8.0)
    if zeros:
        np.testing.assert_array_equal(npi(z), zero.astype(np.uint8))
    code = np.where(sf[:, None] > 0, np.clip(np.rint(v / safe[:, None]) + zero[:, None], 0, 15), zero[:, None])
    got = np.ascontiguousarray(npi(q)).view(np.uint32)
    codes = np.stack([(got >> np.uint32(4 * i)) & np.uint32(15) for i in range(8)], 1).reshape(-1, group, N)
    np.testing.assert_array_equal(codes, code.astype(np.uint32))
    back = f64(moe.w4_dequantize(q, s, z)).reshape(v.shape)
    assert (np.abs(back - v) <= (1.0 if zeros else 0.5) * 1.05 * sf[:, None] + 2.0 ** -8 * np.abs(v)).all()
    moe.sync_status()


def test_bad_ids_are_reported():
    moe = lib()
    T, H, E, k, I, group = 4, 128, 4, 2, 64, 64
    qg, qd = dev_of(*weights(1, E, H, 2 * I, group, False)), dev_of(*weights(2, E, I, H, group, False))
    x = rows_of(1, T, H).to(dev())
    ids = i32(ids_of(3, T, E, k))
    good = moe.w4_gate_up_swiglu(x, ids, *qg)
    for bad in (E, -2, 2 ** 31 - 1):
        wrong = ids.clone()
        wrong[1, 1] = bad
        h = moe.w4_gate_up_swiglu(x, wrong, *qg)
        with pytest.raises(moe.MoEError):
            moe.sync_status()
        assert torch.equal(h[0], good[0]) and float(h[1, 1].float().abs().max()) == 0
        moe.w4_down_combine(h, wrong, None, *qd)
        with pytest.raises(moe.MoEError):
            moe.sync_status()
    moe.sync_status()


@pytest.mark.parametrize("T", [2, 200])
def test_a_wait_that_runs_out_is_reported(T):
    """With no copies issued, the bounded waits (of the kernel of few slots, and
    of the other) give up, the status says so, the context stays usable and the
    next call is right."""
    moe = lib()
    H, E, k, I, group = 256, 4, 2, 128, 64
    qg, qd = dev_of(*weights(1, E, H, 2 * I, group, False)), dev_of(*weights(2, E, I, H, group, True))
    x = rows_of(1, T, H).to(dev())
    ids = i32(ids_of(3, T, E, k))
    h0 = moe.w4_gate_up_swiglu(x, ids, *qg)
    y0 = moe.w4_down_combine(h0, ids, None, *qd)
    moe.set_wait_limit_ns(20_000_000)
    try:
        for call in (lambda: moe.w4_gate_up_swiglu(x, ids, *qg), lambda: moe.w4_down_combine(h0, ids, None, *qd)):
            moe._lib.call("moe_test_stall_gemm_producer", 1)
            call()
            moe._lib.call("moe_test_stall_gemm_producer", 0)
            with pytest.raises(moe.MoEError) as err:
                moe.sync_status()
            assert err.value.status == 4
    finally:
        moe._lib.call("moe_test_stall_gemm_producer", 0)
        moe.set_wait_limit_ns(0)
    assert torch.equal(moe.w4_gate_up_swiglu(x, ids, *qg), h0)
    assert torch.equal(moe.w4_down_combine(h0, ids, None, *qd), y0)
    moe.sync_status()


def test_refusals():
    moe = lib()
    T, H, E, k, I, group = 4, 128, 4, 2, 64, 64
    q, s, _ = dev_of(*weights(1, E, H, 2 * I, group, False))
    x = rows_of(1, T, H).to(dev())
    ids = i32(ids_of(3, T, E, k))
    z = torch.zeros(s.shape, dtype=torch.uint8, device=dev())
    for call in (lambda: moe.w4_gate_up_swiglu(x[:, :120].contiguous(), ids, q, s),       # H and qweight disagree
                 lambda: moe.w4_gate_up_swiglu(x, ids[:3].contiguous(), q, s),
                 lambda: moe.w4_gate_up_swiglu(x, None, q, s),                            # four experts, no ids
                 lambda: moe.w4_gate_up_swiglu(x, ids, q, s[:, :64].contiguous()),
                 lambda: moe.w4_gate_up_swiglu(x, ids, q, s, z[:2]),
                 lambda: moe.w4_gate_up_swiglu(x.t(), ids, q, s),
                 lambda: moe.w4_gate_up_swiglu(x.cpu(), ids, q, s),
                 lambda: moe.w4_quantize(rows_of(1, 96, 64).to(dev()), 64),
                 lambda: moe.w4_down_combine(x.view(T, 1, H), ids, None, q, s)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.w4_gate_up_swiglu(x.float(), ids, q, s), lambda: moe.w4_gate_up_swiglu(x, ids.long(), q, s),
                 lambda: moe.w4_gate_up_swiglu(x, ids, q, s.float()), lambda: moe.w4_gate_up_swiglu(x, ids, q, s, z.int())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: moe.w4_gate_up_swiglu(x, ids, q, s[:4].contiguous()),            # group 128 = H: fine
                 ):
        call()
    with pytest.raises(moe.MoEError):
        moe.w4_gate_up_swiglu(x, ids, q, torch.zeros((E * H // 16, 2 * I), dtype=torch.bfloat16, device=dev()))
    with pytest.raises(moe.MoEError):   # I not a multiple of 64
        moe.w4_gate_up_swiglu(x, ids, q[:, :96].contiguous(), s[:, :96].contiguous())
    moe.sync_status()
