"""Argument checks of the layer for a few tokens, the norms around a block and
the gradients' clipping on the host (CPU only: an invalid call is refused
before any CUDA call)."""
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


def experts(lib, x=FAKE, ids=FAKE, w=FAKE, gu=FAKE, dn=FAKE, sgu=None, sdn=None, T=4, H=128, E=8, k=2, I=64, I_s=0, y=FAKE,
            ws=FAKE, n=1 << 40):
    return lib.moe_few_experts(x, ids, w, gu, dn, sgu, sdn, T, H, E, k, I, I_s, y, ws, n, None)


def test_few_experts(lib):
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(gu=None), dict(dn=None), dict(y=None), dict(x=ODD), dict(gu=ODD),
               dict(dn=ODD), dict(y=ODD), dict(T=-1), dict(H=0), dict(E=0), dict(k=0), dict(I=0), dict(I_s=-64), dict(I_s=64),
               dict(sgu=FAKE, sdn=FAKE), dict(sgu=FAKE, I_s=64), dict(sdn=FAKE, I_s=64), dict(sgu=ODD, sdn=FAKE, I_s=64)):
        assert experts(lib, **kw) == INVALID, kw
    for kw in (dict(H=96), dict(I=96), dict(I_s=96, sgu=FAKE, sdn=FAKE), dict(E=1025), dict(E=64, k=33), dict(T=129, k=1),
               dict(H=2 ** 21), dict(I=2 ** 21), dict(E=1024, H=2 ** 21 + 64), dict(E=1024, I=2 ** 20 - 64, H=2 ** 21)):
        assert experts(lib, **kw) == UNSUPPORTED, kw
    n = ctypes.c_size_t(0)
    assert lib.moe_few_experts_workspace_size(4, 128, 8, 2, 64, 0, ctypes.byref(n)) == 0 and n.value > 0
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=n.value - 1)):
        assert experts(lib, **kw) == WORKSPACE, kw
    assert lib.moe_few_experts_workspace_size(4, 128, 8, 2, 64, 0, None) == INVALID
    assert lib.moe_few_experts_workspace_size(4, 96, 8, 2, 64, 0, ctypes.byref(n)) == UNSUPPORTED
    assert experts(lib, T=0, x=None, ids=None, w=None, y=None, ws=None, n=0) == 0


def layer(lib, x=FAKE, wr=FAKE, bias=None, bal=None, gu=FAKE, dn=FAKE, T=4, H=128, E=8, k=2, I=64, score=0, groups=1, top=1,
          gs=0, renorm=1, scale=1.0, ids=FAKE, w=FAKE, y=FAKE, ws=FAKE, n=1 << 40):
    return lib.moe_few_layer(x, wr, bias, bal, gu, dn, None, None, T, H, E, k, I, 0, score, groups, top, gs, renorm, scale, ids,
                             w, y, ws, n, None)


def test_few_layer(lib):
    for kw in (dict(x=None), dict(wr=None), dict(gu=None), dict(ids=None), dict(w=None), dict(y=None), dict(wr=ODD), dict(bias=ODD),
               dict(bal=ODD), dict(k=9), dict(groups=0), dict(groups=3), dict(top=2), dict(groups=4, top=1, k=3), dict(score=2),
               dict(gs=-1), dict(scale=NAN), dict(scale=INF), dict(T=-1)):
        assert layer(lib, **kw) == INVALID, kw
    for kw in (dict(E=1025), dict(T=129, k=1), dict(H=96), dict(E=128, groups=64, top=64)):
        assert layer(lib, **kw) == UNSUPPORTED, kw
    n = ctypes.c_size_t(0)
    assert lib.moe_few_layer_workspace_size(4, 128, 8, 2, 64, 0, ctypes.byref(n)) == 0
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=n.value - 1)):
        assert layer(lib, **kw) == WORKSPACE, kw
    assert layer(lib, T=0, x=None, ids=None, w=None, y=None, ws=None, n=0) == 0


def norm(lib, x=FAKE, y=FAKE, w=FAKE, v=None, g=None, types=0, T=4, H=64, gates=0, a=1.0, b=1.0, eps=1e-6, r=FAKE, h=FAKE,
         stats=None):
    return lib.moe_block_norm(x, y, w, v, g, types, T, H, gates, a, b, eps, r, h, stats, None)


def test_block_norm(lib):
    for kw in (dict(x=None), dict(y=None, w=None, r=None, h=None), dict(r=None), dict(h=None), dict(w=None), dict(y=None),
               dict(y=None, r=None, v=FAKE), dict(y=None, r=None, g=FAKE, gates=1), dict(y=None, r=None, a=0.5),
               dict(y=None, r=None, b=0.5), dict(x=ODD), dict(y=ODD), dict(w=ODD), dict(v=ODD), dict(g=ODD, gates=1), dict(r=ODD),
               dict(h=ODD), dict(g=FAKE, gates=0), dict(g=None, gates=1), dict(g=FAKE, gates=3), dict(gates=-1), dict(T=-1),
               dict(H=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(a=NAN), dict(b=INF), dict(T=2 ** 31)):
        assert norm(lib, **kw) == INVALID, kw
    for kw in (dict(H=60), dict(H=8200)):
        assert norm(lib, **kw) == UNSUPPORTED, kw
    assert norm(lib, T=0, x=None, y=None, r=None, h=None) == 0


def norm_bwd(lib, dh=FAKE, dr=None, x=FAKE, y=FAKE, stats=FAKE, w=FAKE, v=None, g=None, types=0, T=4, H=64, gates=0, a=1.0, b=1.0,
             dx=FAKE, dy=FAKE, dw=FAKE, dv=None, dg=None, ws=FAKE, n=1 << 40):
    return lib.moe_block_norm_bwd(dh, dr, x, y, stats, w, v, g, types, T, H, gates, a, b, dx, dy, dw, dv, dg, ws, n, None)


def test_block_norm_bwd(lib):
    for kw in (dict(dh=None), dict(x=None), dict(stats=None), dict(dx=None), dict(dy=None), dict(dw=None), dict(dv=FAKE),
               dict(v=FAKE), dict(dg=FAKE), dict(g=FAKE, gates=2), dict(w=None, dw=None), dict(dh=ODD), dict(dr=ODD), dict(dx=ODD),
               dict(dy=ODD), dict(dw=ODD), dict(y=None, a=2.0), dict(y=None), dict(g=FAKE, dg=FAKE, gates=3), dict(a=INF)):
        assert norm_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(H=60), dict(H=8200)):
        assert norm_bwd(lib, **kw) == UNSUPPORTED, kw
    n = ctypes.c_size_t(0)
    assert lib.moe_block_norm_bwd_workspace_size(4, 64, 0, 1, 0, ctypes.byref(n)) == 0 and n.value > 0
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=n.value - 1)):
        assert norm_bwd(lib, **kw) == WORKSPACE, kw
    for args in ((-1, 64, 0), (4, 0, 0), (4, 64, -1)):
        assert lib.moe_block_norm_bwd_workspace_size(*args, 1, 0, ctypes.byref(n)) == INVALID
    assert lib.moe_block_norm_bwd_workspace_size(4, 64, 0, 1, 0, None) == INVALID


def clip(lib, grads=(0x10000,), outs=(0x10000,), sizes=(8,), f32=(1,), max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE, n=1 << 40):
    arr = lambda t, v: None if v is None else (t * max(len(v), 1))(*v)
    return lib.moe_grad_clip(arr(P, grads), arr(P, outs), arr(ctypes.c_int64, sizes), arr(ctypes.c_uint8, f32), len(sizes), max_norm,
                             eps, norm, ws, n, None)


def test_grad_clip(lib):
    for kw in (dict(grads=None), dict(f32=None), dict(grads=(None,)), dict(outs=(None,)), dict(grads=(0x10002,)), dict(outs=(0x10002,)),
               dict(grads=(0x10001,), f32=(0,)), dict(sizes=(-1,)), dict(sizes=(2 ** 45,)), dict(max_norm=-1.0), dict(max_norm=NAN),
               dict(eps=-1.0), dict(eps=NAN), dict(norm=None)):
        assert clip(lib, **kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=7)):
        assert clip(lib, **kw) == WORKSPACE, kw
    n = ctypes.c_size_t(0)
    sizes, f32 = (ctypes.c_int64 * 2)(2 ** 14, 2 ** 14 + 1), (ctypes.c_uint8 * 2)(1, 1)
    grads = (P * 2)(0x10000, 0x10004)
    assert lib.moe_grad_clip_workspace_size(grads, sizes, f32, 2, ctypes.byref(n)) == 0 and n.value == 8 * 2
    assert lib.moe_grad_clip_workspace_size(grads, sizes, f32, 2, None) == INVALID
