"""Argument checks of the expert choice and of the 4-bit experts on the host
(CPU only: an invalid call is refused before any CUDA call)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = P(0x10000)       # a 16-byte aligned non-null pointer; never dereferenced on these paths
ODD = P(0x10002)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    import token_dispatch_grouped_softmax_gb300 as moe

    moe.build()
    return moe.load()


def select(lib, logits=FAKE, bias=None, T=4, E=16, k=2, score=0, groups=1, top=1, gs=0, renorm=1, scale=1.0, ids=FAKE, w=FAKE):
    return lib.moe_route_select(logits, 0, bias, T, E, k, score, groups, top, gs, renorm, scale, ids, w, None)


def test_route_select(lib):
    for kw in (dict(k=0), dict(k=17), dict(E=0), dict(T=-1), dict(T=2 ** 31), dict(groups=3), dict(groups=0),
               dict(groups=4, top=5), dict(groups=4, top=0), dict(groups=4, top=1, k=5), dict(score=2), dict(score=-1),
               dict(gs=2), dict(scale=NAN), dict(scale=INF), dict(logits=None), dict(ids=None), dict(w=None),
               dict(logits=ODD), dict(bias=ODD), dict(T=2 ** 30, k=4)):
        assert select(lib, **kw) == INVALID, kw
    assert select(lib, E=2048) == UNSUPPORTED
    assert select(lib, E=64, k=33) == UNSUPPORTED
    assert select(lib, E=128, groups=64, top=64) == UNSUPPORTED
    assert select(lib, T=0, logits=None, ids=None, w=None) == 0


def bwd(lib, dw=FAKE, nparts=1, row_map=None, logits=FAKE, ids=FAKE, T=4, E=16, k=2, score=0, renorm=1, scale=1.0, out=FAKE):
    return lib.moe_route_select_bwd(dw, nparts, row_map, logits, 0, ids, T, E, k, score, renorm, scale, out, None, None)


def test_route_select_bwd_and_balance_bias(lib):
    for kw in (dict(nparts=0), dict(k=0), dict(k=17), dict(score=5), dict(scale=INF), dict(dw=None), dict(logits=None),
               dict(ids=None), dict(out=None), dict(logits=ODD), dict(out=ODD)):
        assert bwd(lib, **kw) == INVALID, kw
    assert bwd(lib, E=1025) == UNSUPPORTED
    assert bwd(lib, T=0, dw=None, logits=None, ids=None, out=None) == 0
    b = lib.moe_route_balance_bias
    for args in ((None, FAKE, 8, 0.1, FAKE), (FAKE, None, 8, 0.1, FAKE), (FAKE, FAKE, 8, 0.1, None), (FAKE, FAKE, 0, 0.1, FAKE),
                 (FAKE, FAKE, 8, NAN, FAKE)):
        assert b(*args, None) == INVALID
    assert b(FAKE, FAKE, 1025, 0.1, FAKE, None) == UNSUPPORTED


def gate_up(lib, x=FAKE, ids=FAKE, q=FAKE, s=FAKE, z=None, T=4, H=128, E=8, k=2, I=64, group=64, h=FAKE):
    return lib.moe_w4_gate_up_swiglu(x, ids, q, s, z, T, H, E, k, I, group, h, None)


def test_w4_gate_up(lib):
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(h=None), dict(x=ODD), dict(q=ODD), dict(s=ODD), dict(z=ODD),
               dict(h=ODD), dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(I=0), dict(ids=None), dict(T=2 ** 30, k=4)):
        assert gate_up(lib, **kw) == INVALID, kw
    for kw in (dict(group=16), dict(group=256), dict(H=96), dict(H=192, group=128), dict(I=32), dict(E=1025, k=2),
               dict(E=64, k=33), dict(H=2 ** 21), dict(I=2 ** 20)):
        assert gate_up(lib, **kw) == UNSUPPORTED, kw
    assert gate_up(lib, T=0, x=None, ids=None, h=None) == 0


def down(lib, h=FAKE, ids=FAKE, w=None, q=FAKE, s=FAKE, z=None, ys=None, T=4, H=128, E=8, k=2, I=64, group=64, y=FAKE, ws=FAKE,
         n=1 << 30):
    return lib.moe_w4_down_combine(h, ids, w, q, s, z, ys, T, H, E, k, I, group, y, ws, n, None)


def test_w4_down(lib):
    for kw in (dict(h=None), dict(y=None), dict(h=ODD), dict(y=ODD), dict(ys=ODD), dict(z=ODD), dict(ids=None), dict(k=9)):
        assert down(lib, **kw) == INVALID, kw
    for kw in (dict(H=96), dict(I=96), dict(I=64, group=128), dict(group=8), dict(E=1025), dict(I=2 ** 21), dict(H=2 ** 21)):
        assert down(lib, **kw) == UNSUPPORTED, kw
    n = ctypes.c_size_t(0)
    assert lib.moe_w4_down_workspace_size(4, 128, 2, ctypes.byref(n)) == 0 and n.value >= 4 * 2 * 128 * 4
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=n.value - 1)):
        assert down(lib, **kw) == WORKSPACE, kw
    assert lib.moe_w4_down_workspace_size(4, 128, 2, None) == INVALID
    assert down(lib, T=0, h=None, ids=None, y=None, ws=None, n=0) == 0


def test_w4_quantize(lib):
    for f in (lib.moe_w4_quantize, lambda w, r, n, g, q, s, z, st: lib.moe_w4_dequantize(q, s, z, r, n, g, w, st)):
        for args in ((None, 128, 64, 64, FAKE, FAKE, None), (FAKE, 128, 64, 64, None, FAKE, None),
                     (FAKE, 128, 64, 64, FAKE, None, None), (FAKE, 0, 64, 64, FAKE, FAKE, None),
                     (ODD, 128, 64, 64, FAKE, FAKE, None), (FAKE, 128, 64, 64, FAKE, FAKE, ODD)):
            assert f(*args, None) == INVALID, args
        for args in ((FAKE, 128, 32, 64, FAKE, FAKE, None), (FAKE, 96, 64, 64, FAKE, FAKE, None),
                     (FAKE, 128, 64, 48, FAKE, FAKE, None)):
            assert f(*args, None) == UNSUPPORTED, args
