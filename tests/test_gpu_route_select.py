"""The expert choice (moe_route_select), its gradient and the balance bias on
the GPU against 64-bit references."""
import numpy as np
import pytest
import torch

import ref_select as ref
from gpu_helpers import dev, f32, f64, i32, lib, npi

pytestmark = pytest.mark.gpu
U = ref.U


def logits_of(seed, T, E, dtype=torch.float32, masked=0.0, spread=1.5):
    g = np.random.default_rng(seed)
    z = torch.from_numpy((spread * g.normal(size=(T, E))).astype(np.float32)).to(dtype)
    if masked:
        z[torch.from_numpy(g.random((T, E)) < masked)] = -float("inf")
    return z.to(dev())


CASES = [  # T, E, k, n_groups, top_groups, group_score
    (1, 8, 2, 1, 1, "max"), (7, 60, 5, 6, 3, "max"), (33, 60, 4, 4, 2, "top2"), (130, 128, 8, 1, 1, "max"),
    (64, 256, 8, 8, 4, "top2"), (9, 256, 8, 8, 8, "top2"), (5, 1024, 32, 1, 1, "max"), (6, 1024, 17, 32, 9, "top2"),
    (11, 96, 6, 3, 1, "top2"), (4, 1020, 6, 17, 5, "max"), (3, 32, 3, 32, 3, "top2"), (21, 12, 12, 3, 3, "max"),
    (17, 1, 1, 1, 1, "max"), (10, 510, 9, 2, 1, "top2")]


@pytest.mark.parametrize("T,E,k,groups,top,gs", CASES)
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("bias", (False, True))
def test_choice_and_weights(T, E, k, groups, top, gs, score, bias):
    """Ids are the reference's wherever its compared values are not within
    fp32's reach of each other (16 U of 1 + |bias|, the largest a value gets);
    the weights are those of the ids.  Their bound: expf 2 ulp = 4 U, the
    exponent's own rounding |z - m| U, the sums' k (or E) U, and a few U for
    the quotients and the scale."""
    moe = lib()
    for dtype, renorm, scale in ((torch.float32, True, 1.0), (torch.float32, False, 2.5), (torch.bfloat16, True, 2.5)):
        z = logits_of(T + E + k, T, E, dtype)
        b = 0.2 * np.random.default_rng(E).normal(size=E).astype(np.float32) if bias else None
        how = dict(score=score, n_groups=groups, top_groups=top, group_score=gs, renorm=renorm, scale=scale)
        ids, w = moe.route_select(z, k, bias=None if b is None else f32(b), **how)
        moe.sync_status()
        z64 = f64(z)
        r = ref.select(z64, k, bias=b, **how)
        near = 0 < r["gap"]
        near &= r["gap"] < 16 * U * 2.0 * (1.0 + (np.abs(b).max() if bias else 0.0))
        same = (npi(ids) == r["ids"]).all(1)
        assert (same | near).all()
        assert near.sum() <= 1 + T // 50
        assert all(len(set(row)) == k for row in npi(ids).tolist())
        spread = z64.max() - z64.min()
        np.testing.assert_allclose(f64(w), ref.weights_of(z64, npi(ids).astype(np.int64), score, renorm, scale),
                                   rtol=(16 + E + k + spread) * 2 * U, atol=1e-37)


def test_equal_values_go_to_the_lower_index():
    """Logits on a coarse grid (many exact ties among experts and groups), -0
    equal to +0, in every group shape."""
    moe = lib()
    g = np.random.default_rng(5)
    for T, E, k, groups, top, gs in CASES:
        z = np.round(g.normal(size=(T, E))).astype(np.float32)
        z[z == 0] = np.where(g.random((z == 0).sum()) < 0.5, -0.0, 0.0)
        ids, _ = moe.route_select(f32(z), k, n_groups=groups, top_groups=top, group_score="max", score="sigmoid")
        r = ref.select(z, k, score="sigmoid", n_groups=groups, top_groups=top, group_score="max")
        np.testing.assert_array_equal(npi(ids), r["ids"])
    # values that tie only after the bias: sigmoid(0) = 1/2 and a bias in halves
    z = np.zeros((2, 16), np.float32)
    b = np.tile(np.array([0.0, 0.5, 0.5, 0.25], np.float32), 4)
    ids, w = moe.route_select(f32(z), 4, bias=f32(b), score="sigmoid", n_groups=4, top_groups=2)
    assert npi(ids).tolist() == [[1, 2, 5, 6]] * 2
    np.testing.assert_array_equal(f64(w), 0.25)


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("bias", (False, True))
@pytest.mark.parametrize("renorm", (False, True))
def test_masked_experts(score, bias, renorm):
    """Logits of -inf: never chosen before an unmasked expert of the chosen
    groups, weight 0; whole groups and whole rows masked; the gradient is 0
    there and finite everywhere."""
    moe = lib()
    T, E, k = 40, 32, 6
    z = logits_of(9, T, E, masked=0.8)
    z[0] = -float("inf")
    z[1, 4:] = -float("inf")
    z[2, :8] = -float("inf")
    b = np.random.default_rng(1).normal(size=E).astype(np.float32) if bias else None
    for groups, top, gs in ((1, 1, "max"), (4, 2, "top2"), (4, 1, "max"), (8, 3, "top2")):
        kk = min(k, top * E // groups)
        how = dict(score=score, n_groups=groups, top_groups=top, group_score=gs, renorm=renorm)
        ids, w = moe.route_select(z, kk, bias=None if b is None else f32(b), **how)
        z64 = f64(z)
        r = ref.select(z64, kk, bias=b, **how)
        np.testing.assert_array_equal(npi(ids), r["ids"])
        np.testing.assert_allclose(f64(w), r["w"], rtol=2e-5, atol=1e-37)
        assert (f64(w)[0] == 0).all()
        dw = f32(np.random.default_rng(2).normal(size=(T, kk)))
        d = f64(moe.route_select_bwd(dw, z, ids, score=score, renorm=renorm))
        assert np.isfinite(d).all() and (d[np.isneginf(z64)] == 0).all()
        np.testing.assert_allclose(d, ref.select_bwd(f64(dw), z64, r["ids"], score, renorm, 1.0), atol=2e-5)
    moe.sync_status()


@pytest.mark.parametrize("E,k", [(256, 8), (60, 5), (250, 32), (32, 32)])
@pytest.mark.parametrize("low,high", [(-110.0, 110.0), (-90.0, -70.0), (4.0, 20.0), (-1.0, 1.0)])
def test_sigmoid_scores_are_the_rounded_steps(E, k, low, high):
    """1 / (1 + exp(-z)), each step rounded to fp32, bit for bit: nearly equal
    and saturated scores choose the experts that they choose, and the weights
    are those scores, subnormal ones too."""
    moe = lib()
    rng = np.random.default_rng(E)
    z = f32(rng.uniform(low, high, (700, E)))
    z[::7, 3] = float("-inf")
    s = 1 / (1 + torch.exp(-z))
    zero = torch.zeros(E, device=dev())
    ids, w = moe.route_select(z, k, bias=zero, score="sigmoid", renorm=False)
    value = torch.where(z == float("-inf"), torch.full_like(s, float("-inf")), s)
    want = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    assert torch.equal(w, s.gather(1, want))
    ids2, w2 = moe.route_select(z, k, score="sigmoid", renorm=False)   # chosen by the logits
    assert torch.equal(w2, s.gather(1, ids2.long()))
    moe.sync_status()


def test_nan_and_infinite_logits():
    """A NaN is chosen first and its weight is NaN; ids stay distinct and in
    range; the other rows are untouched."""
    moe = lib()
    z = logits_of(3, 6, 64)
    clean = z.clone()
    z[2, 17] = float("nan")
    z[4, 5] = float("inf")
    for score in ("softmax", "sigmoid"):
        ids, w = moe.route_select(z, 4, score=score, n_groups=4, top_groups=2, group_score="max")
        ids0, w0 = moe.route_select(clean, 4, score=score, n_groups=4, top_groups=2, group_score="max")
        keep = [0, 1, 3, 5]
        assert torch.equal(ids[keep], ids0[keep]) and torch.equal(w[keep], w0[keep])
        assert int(ids[2, 0]) == 17 and bool(w[2].isnan().any()) and int(ids[4, 0]) == 5
        assert all(len(set(r)) == 4 and 0 <= min(r) and max(r) < 64 for r in npi(ids).tolist())


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (33, 60, 5), (130, 128, 8), (6, 1024, 32), (5, 7, 1), (9, 256, 8)])
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
def test_gradient(T, E, k, score, renorm):
    """Against the chain rule and against central differences of the 64-bit
    forward (h = 1e-4: error 10 h^2).  Each term scale * s_j * dw carries the
    relative bound of the forward's weights, on the sum of the terms'
    magnitudes; bf16 results add half an ulp."""
    moe = lib()
    scale = 2.5
    for dtype in (torch.float32, torch.bfloat16):
        z = logits_of(E + k, T, E, dtype)
        z64 = f64(z)
        dw = np.random.default_rng(T).normal(size=(T, k)).astype(np.float32)
        ids, _ = moe.route_select(z, k, score=score, renorm=renorm, scale=scale)
        d = moe.route_select_bwd(f32(dw), z, ids, score=score, renorm=renorm, scale=scale)
        moe.sync_status()
        assert d.dtype == dtype
        i64 = npi(ids).astype(np.int64)
        r = ref.select_bwd(dw, z64, i64, score, renorm, scale)
        s = ref.scores(z64, score)
        spread = z64.max() - z64.min()
        mag = scale * np.abs(dw).sum(1, keepdims=True) * (s if not renorm else np.ones_like(s))
        tol = (24 + E + k + spread) * 2 * U * mag + 1e-37
        if dtype == torch.bfloat16:
            tol = tol + ref.half_ulp_bf16(np.abs(r) + tol)
        assert (np.abs(f64(d) - r) <= tol).all()
        h = 1e-4
        for e in np.random.default_rng(E).choice(E, min(E, 6), replace=False):
            zp, zm = z64.copy(), z64.copy()
            zp[:, e] += h
            zm[:, e] -= h
            diff = ((ref.weights_of(zp, i64, score, renorm, scale) -
                     ref.weights_of(zm, i64, score, renorm, scale)) * dw).sum(1) / (2 * h)
            assert (np.abs(f64(d)[:, e] - diff) <= tol[:, e] + 10 * scale * k * 4 * h * h).all()


def test_gradient_from_partials():
    """dw summed from the down backward's partials through row_map equals the
    gradient of the summed dw, and route_bwd's dw bit for bit."""
    moe = lib()
    T, E, k, parts = 50, 64, 6, 3
    g = np.random.default_rng(8)
    z = logits_of(8, T, E)
    ids, w = moe.route_select(z, k)
    row_map = i32(g.permutation(T * k))
    part = f32(g.normal(size=(T * k, parts)))
    d, dw = moe.route_select_bwd(part, z, ids, row_map=row_map)
    d0, dw0 = moe.route_bwd(part, row_map, w, ids, E)
    assert torch.equal(dw, dw0)
    assert torch.equal(d, moe.route_select_bwd(dw, z, ids))
    # the same formula on w rounded in another place: w's bound on each factor
    assert float((d - d0).abs().max()) <= 64 * 2 * U * float(dw.abs().sum(1).max())
    moe.sync_status()


def test_bad_device_data_is_reported():
    moe = lib()
    z = logits_of(1, 4, 16)
    ids, _ = moe.route_select(z, 2)
    dw = torch.ones((4, 2), device=dev())
    bad = ids.clone()
    bad[1, 0] = 16
    moe.route_select_bwd(dw, z, bad)
    with pytest.raises(moe.MoEError):
        moe.sync_status()
    rows = torch.arange(8, dtype=torch.int32, device=dev())
    rows[3] = 99
    moe.route_select_bwd(torch.ones((8, 1), device=dev()), z, ids, row_map=rows)
    with pytest.raises(moe.MoEError):
        moe.sync_status()
    moe.sync_status()


@pytest.mark.parametrize("E", (1, 8, 60, 1024))
def test_balance_bias(E):
    """Bit for bit: the sign from integers (experts at the mean keep their
    bias), loads whose sum passes 32 bits, in place."""
    moe = lib()
    g = np.random.default_rng(E)
    counts = g.integers(0, 2 ** 31 - 1 if E > 8 else 4, size=E).astype(np.int32)
    b = g.normal(size=E).astype(np.float32)
    sign = np.sign(counts.astype(object).sum() - E * counts.astype(object)).astype(np.float32)
    want = b + np.float32(0.001) * sign
    bias, c = f32(b), i32(counts)
    out = moe.route_balance_bias(bias, c, 0.001)
    np.testing.assert_array_equal(out.cpu().numpy(), want)
    assert moe.route_balance_bias(bias, c, 0.001, out=bias) is bias and torch.equal(bias, out)


def test_streams_and_empty_batch():
    """On a stream of its own, behind the work that writes its logits; T = 0."""
    moe = lib()
    s = torch.cuda.Stream()
    z = logits_of(4, 4096, 64)
    ref_ids, ref_w = moe.route_select(2 * z, 4)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=dev())
        for _ in range(4):
            big = big @ big * 1e-3
        z2 = z + z
        ids, w = moe.route_select(z2, 4)
        d = moe.route_select_bwd(w, z2, ids)
    s.synchronize()
    assert torch.equal(ids, ref_ids) and torch.equal(w, ref_w)
    assert torch.equal(d, moe.route_select_bwd(ref_w, 2 * z, ref_ids))
    e = torch.empty((0, 64), device=dev())
    ids, w = moe.route_select(e, 4)
    assert ids.shape == (0, 4) and moe.route_select_bwd(w, e, ids).shape == (0, 64)
    moe.sync_status()


def test_a_view_at_an_odd_offset():
    """Logits that start inside another tensor (16-byte aligned rows or not):
    the row stride E need not be a multiple of 4."""
    moe = lib()
    base = logits_of(6, 50, 61)
    view = base[4:]          # 4 * 61 * 4 bytes: 16-byte aligned start
    ids, w = moe.route_select(view, 5)
    ids0, w0 = moe.route_select(view.clone(), 5)
    assert torch.equal(ids, ids0) and torch.equal(w, w0)
    with pytest.raises(moe.MoEError):
        moe.route_select(base[1:], 5)   # 244 bytes: not aligned


def test_refusals():
    moe = lib()
    z = logits_of(1, 4, 16)
    for kw in (dict(k=17), dict(k=0), dict(k=5, n_groups=4, top_groups=1), dict(k=2, n_groups=3), dict(k=2, n_groups=0),
               dict(k=2, n_groups=4, top_groups=5), dict(k=2, scale=float("nan"))):
        k = kw.pop("k")
        with pytest.raises((moe.MoEError, RuntimeError)):
            moe.route_select(z, k, **kw)
    with pytest.raises(moe.MoEError):
        moe.route_select(logits_of(1, 2, 1056), 2)
    with pytest.raises(ValueError):
        moe.route_select(z, 2, score="relu")
    with pytest.raises(ValueError):
        moe.route_select(z, 2, group_score="mean")
    with pytest.raises(ValueError):
        moe.route_select(z, 2, bias=torch.zeros(15, device=dev()))
    with pytest.raises(TypeError):
        moe.route_select(z.half(), 2)
    with pytest.raises(ValueError):
        moe.route_select(z.t(), 2)
    with pytest.raises(ValueError):
        moe.route_select(z.cpu(), 2)
    ids, w = moe.route_select(z, 2)
    with pytest.raises(ValueError):
        moe.route_select_bwd(w[:, :1].contiguous(), z, ids)
    with pytest.raises(ValueError):
        moe.route_balance_bias(torch.zeros(16, device=dev()), torch.zeros(15, dtype=torch.int32, device=dev()), 0.1)
    moe.sync_status()
