"""The norms around a block with its gate and residual, forward and backward,
against the formulas in 64 bits (gradients by autograd, and by differences).

Tolerances, from the arithmetic: u = 2^-24 is fp32's half step.  The sum of
at most 8192 squares in a tree of depth below 32, its root, the division and
the few products and sums of an output come to at most 64 roundings of
quantities no larger than the output's terms taken with positive signs (its
"size"): 64 u = 2^-18 of the size.  A sum over T rows adds T u of the sum of
its terms' sizes.  The output's own rounding is half a step of its type."""
import pytest
import torch

from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(T, H, x="bf16", branch=True, weight="f32", post=None, gates=0, gate="f32", seed=0, scale=3.0):
    g = torch.Generator().manual_seed(1000 * T + H + seed)
    make = lambda shape, t, a=1.0, b=0.0: (b + a * torch.randn(shape, generator=g)).to(t).to(dev())
    d = dict(x=make((T, H), TYPES[x], scale))
    d["branch"] = make((T, H), torch.bfloat16) if branch else None
    d["weight"] = make((H,), TYPES[weight], 0.2, 1.0) if weight else None
    d["post_weight"] = make((H,), TYPES[post], 0.2, 1.0) if post else None
    d["gate"] = make((gates, H), TYPES[gate], 0.5) if gates else None
    up = dict(dh=make((T, H), torch.bfloat16) if weight else None, dr=make((T, H), TYPES[x]) if branch else None)
    return d, up


def model(d, a, b):
    """r and h in 64 bits, from leaves that record gradients."""
    v = {n: None if t is None else t.double().requires_grad_() for n, t in d.items()}
    T, H = d["x"].shape

    def rms(t, w):
        return t / torch.sqrt(t.square().mean(1, keepdim=True) + EPS) * w

    r = v["x"]
    if v["branch"] is not None:
        n = v["branch"] if v["post_weight"] is None else rms(v["branch"], v["post_weight"])
        if v["gate"] is not None:
            n = (n.view(v["gate"].shape[0], -1, H) * v["gate"].unsqueeze(1)).view(T, H)
        r = a * r + b * n
    return v, r, None if v["weight"] is None else rms(r, v["weight"])


def sizes(d, up, a, b):
    """The outputs' formulas with every term positive."""
    p = {n: None if t is None else t.double().abs() for n, t in {**d, **up}.items()}
    one = torch.ones((), dtype=torch.float64, device=dev())
    T, H = p["x"].shape
    get = lambda n: one if p[n] is None else p[n]
    L = T // p["gate"].shape[0] if p["gate"] is not None else 1
    g = get("gate").repeat_interleave(L, 0) if p["gate"] is not None else one
    out = {}
    with torch.no_grad():
        _, r64, _ = model(d, a, b)
        r, sy, y = p["x"], one, None
        if p["branch"] is not None:
            y = p["branch"]
            if p["post_weight"] is not None:
                sy = 1 / torch.sqrt(y.square().mean(1, keepdim=True) + EPS)
            n = y * sy * get("post_weight")
            r = abs(a) * p["x"] + abs(b) * g * n
            out["r"] = r
        sr = 1 / torch.sqrt(r64.square().mean(1, keepdim=True) + EPS)
        # r's own error carries into the statistics of its row
        spread = (r * r64.abs()).mean(1, keepdim=True) * sr * sr
        xn = r * sr + r64.abs() * sr * spread
        if p["weight"] is not None:
            out["h"] = xn * p["weight"]
        dd = torch.zeros_like(p["x"]) if p["dr"] is None else p["dr"]
        if p["weight"] is not None:
            t = p["dh"] * p["weight"]
            dd = dd + sr * (1 + spread) * (t + xn * (t * xn).mean(1, keepdim=True))
            out["d_weight"] = (p["dh"] * xn).sum(0)
        out["dx"] = abs(a) * dd
        if y is not None:
            dn = abs(b) * dd
            if p["gate"] is not None:
                out["d_gate"] = (dn * n).view(-1, L, H).sum(1)
            dn = dn * g
            if p["post_weight"] is not None:
                out["d_post_weight"] = (dn * y * sy).sum(0)
                t = dn * p["post_weight"]
                dn = sy * (t + y * sy * (t * y * sy).mean(1, keepdim=True))
            out["d_branch"] = dn
    return out


def check(name, got, ref, size, rows=0):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    allow = (1 + half) * (2.0 ** -18 + rows * 2.0 ** -24) * size + half * ref.abs() + 1e-38
    worst = (err - allow).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, (name, worst, err.max().item())


def run_both(moe, d, up, a=1.0, b=1.0):
    T = d["x"].shape[0]
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"], residual_scale=a, branch_scale=b)
    r, h, stats = moe.block_norm(d["x"], eps=EPS, save_for_backward=True, **kw)
    grads = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw)
    size = sizes(d, up, a, b)
    v, r64, h64 = model(d, a, b)
    pairs = [(o, g.double()) for o, g in ((r64 if r is not None else None, up["dr"]), (h64, up["dh"])) if o is not None and g is not None]
    torch.autograd.backward([o for o, _ in pairs], [g for _, g in pairs])
    if r is not None:
        check("r", r, r64.detach(), size["r"])
    if h is not None:
        check("h", h, h64.detach(), size["h"])
    check("dx", grads["dx"], v["x"].grad, size["dx"])
    for mine, leaf, rows in (("d_branch", "branch", 0), ("d_weight", "weight", T), ("d_post_weight", "post_weight", T), ("d_gate", "gate", T)):
        if d[leaf] is None:
            assert grads[mine] is None
        else:
            assert grads[mine].dtype == d[leaf].dtype
            check(mine, grads[mine], v[leaf].grad, size[mine], rows)
    moe.sync_status()
    return r, h, stats, grads


@pytest.mark.parametrize("H", (8, 64, 248, 256, 264, 1000, 2048, 2056, 4104, 7168, 8192))
@pytest.mark.parametrize("T", (1, 2, 7, 200))
def test_sizes(T, H):
    d, up = inputs(T, H, post="f32", gates=1)
    run_both(lib(), d, up)


@pytest.mark.parametrize("kw", (dict(branch=False), dict(branch=False, x="f32", weight="bf16"), dict(weight=None), dict(weight=None, x="f32"),
                                dict(weight=None, post="bf16"), dict(x="f32", post="f32"), dict(weight="bf16", post="bf16", gates=1, gate="bf16"),
                                dict(x="f32", post="bf16", gates=1), dict(gates=1), dict(weight=None, gates=1), dict()))
@pytest.mark.parametrize("T,H", ((33, 96), (700, 512)))
def test_operands(T, H, kw):
    d, up = inputs(T, H, **kw)
    run_both(lib(), d, up, *((1.0, 1.0) if d["branch"] is None else (0.7, 0.22)))


@pytest.mark.parametrize("T,gates", ((6, 2), (6, 3), (6, 6), (640, 4), (640, 320), (640, 640), (5000, 10), (5000, 1250), (4999, 4999), (1217, 1217),
                                     (1500, 500), (1216, 608)))
@pytest.mark.parametrize("H", (64, 320, 2048))
def test_gates(T, gates, H):
    """Groups that end inside a block's rows, span several blocks, or are single rows."""
    d, up = inputs(T, H, post="f32" if gates % 2 else None, gates=gates, gate="bf16" if T % 2 else "f32")
    run_both(lib(), d, up, 1.0, 0.5)


@pytest.mark.parametrize("T", (3000, 16384))
def test_many_rows(T):
    d, up = inputs(T, 1024, post="f32", gates=1)
    run_both(lib(), d, up)


def test_without_dr():
    """A block whose residual is used no further: dr None is a dr of zeros."""
    moe = lib()
    d, up = inputs(40, 256, post="f32", gates=2)
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])
    _, _, stats = moe.block_norm(d["x"], save_for_backward=True, **kw)
    a = moe.block_norm_bwd(up["dh"], None, d["x"], stats, **kw)
    b = moe.block_norm_bwd(up["dh"], torch.zeros_like(d["x"]), d["x"], stats, **kw)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_zero_large_and_special_rows():
    """Rows of zeros, tiny, large, and with an infinity or NaN, which stay in their row."""
    moe = lib()
    d, up = inputs(9, 512, post="f32")
    for n, row in (("x", 1), ("branch", 1), ("branch", 2)):
        d[n][row] = 0
    d["x"][3] *= 1e-20
    d["branch"][3] *= 1e-20
    d["x"][4] *= 1e15
    d["branch"][5] *= 1e15
    run_both(moe, d, up)
    clean = moe.block_norm(d["x"], d["weight"], d["branch"], d["post_weight"])
    d["x"][7, 3] = float("inf")
    d["branch"][8, 500] = float("nan")
    r, h, _ = moe.block_norm(d["x"], d["weight"], d["branch"], d["post_weight"])
    assert torch.equal(r[:7], clean[0][:7]) and torch.equal(h[:7], clean[1][:7])
    assert torch.isinf(r[7, 3]) and torch.isfinite(r[7, 4:]).all() and torch.isnan(h[7]).any() and torch.isnan(h[8]).all()


def test_a_row_does_not_depend_on_the_others():
    moe = lib()
    d, _ = inputs(777, 2048, post="f32", gates=1)
    kw = dict(weight=d["weight"], post_weight=d["post_weight"], gate=d["gate"])
    r, h, _ = moe.block_norm(d["x"], branch=d["branch"], **kw)
    for a, b in ((0, 1), (5, 12), (300, 777)):
        r2, h2, _ = moe.block_norm(d["x"][a:b], branch=d["branch"][a:b], **kw)
        assert torch.equal(r2, r[a:b]) and torch.equal(h2, h[a:b])


def test_the_gradients_are_the_same_every_time():
    moe = lib()
    d, up = inputs(3001, 1024, post="f32", gates=3001)
    d["gate"] = d["gate"][:1].contiguous()
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])
    _, _, stats = moe.block_norm(d["x"], save_for_backward=True, **kw)
    first = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw)
    for _ in range(5):
        again = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_no_rows():
    moe = lib()
    d, up = inputs(0, 64, post="f32")
    d["gate"] = torch.ones((3, 64), device=dev())
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])
    r, h, stats = moe.block_norm(d["x"], save_for_backward=True, **kw)
    assert r.shape == h.shape == (0, 64) and stats.shape == (2, 0)
    g = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw)
    for n in ("d_weight", "d_post_weight", "d_gate"):
        assert bool((g[n] == 0).all())
    assert g["dx"].shape == (0, 64)


def test_by_differences():
    """The gradient along random directions against central differences of the 64-bit model of the kernels' own inputs."""
    moe = lib()
    d, up = inputs(5, 64, x="f32", post="f32", gates=5, seed=3)
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])
    _, _, stats = moe.block_norm(d["x"], save_for_backward=True, **kw)
    g = moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw)
    gen = torch.Generator().manual_seed(11)

    def value(e):
        with torch.no_grad():
            _, r, h = model(e, 1.0, 1.0)
            return float((r * up["dr"].double()).sum() + (h * up["dh"].double()).sum())

    for leaf, grad in (("x", "dx"), ("branch", "d_branch"), ("weight", "d_weight"), ("post_weight", "d_post_weight"), ("gate", "d_gate")):
        way = torch.randn(d[leaf].shape, generator=gen, dtype=torch.float64).to(dev())
        step = 1e-4
        moved = [value({**d, leaf: d[leaf].double() + s * way}) for s in (step, -step)]
        want = (moved[0] - moved[1]) / (2 * step)
        mine = float((g[grad].double() * way).sum())
        # the gradient's rounding along the way, and step^2 of the third derivative (of order 1 here)
        allow = (torch.finfo(g[grad].dtype).eps / 2 + 2.0 ** -16) * float((g[grad].double().abs() * way.abs()).sum()) + 1e-4
        assert abs(mine - want) <= allow, (leaf, mine, want, allow)


def test_in_a_graph_and_on_another_stream():
    moe = lib()
    d, up = inputs(100, 512, post="f32", gates=4)
    kw = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])

    def step():
        r, h, stats = moe.block_norm(d["x"], save_for_backward=True, **kw)
        return dict(r=r, h=h, **moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **kw))

    want = {n: t.clone() for n, t in step().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(other[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    d["x"] += 1
    want = {n: t.clone() for n, t in step().items()}
    graph.replay()
    assert all(torch.equal(out[n], want[n]) for n in want)


@pytest.mark.parametrize("x", ("bf16", "f32"))
def test_in_place(x):
    """The C entry with r the memory of x, at sizes where rows are loaded ahead of the ones that are written."""
    import ctypes

    moe = lib()
    d, _ = inputs(2000, 512, x=x, post="f32", gates=1)
    want = moe.block_norm(d["x"], d["weight"], d["branch"], d["post_weight"], d["gate"])
    h, P = torch.empty_like(want[1]), ctypes.c_void_p
    p = lambda t: P(t.data_ptr())
    types = 2 | 4 | 8 | (1 if x == "f32" else 0)
    rc = moe.load().moe_block_norm(p(d["x"]), p(d["branch"]), p(d["weight"]), p(d["post_weight"]), p(d["gate"]), types, 2000, 512, 1, 1.0, 1.0,
                                   EPS, p(d["x"]), p(h), None, P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and torch.equal(d["x"], want[0]) and torch.equal(h, want[1])
    moe.sync_status()


def test_refusals():
    moe = lib()
    d, up = inputs(12, 64, post="f32", gates=3)
    x, w, y = d["x"], d["weight"], d["branch"]
    for bad in (dict(weight=w[:32]), dict(branch=y[:6]), dict(branch=y.float()), dict(weight=w.half()), dict(gate=d["gate"][:, :32], branch=y),
                dict(gate=torch.ones((5, 64), device=dev()), branch=y), dict(weight=w, post_weight=w), dict(weight=w, residual_scale=0.5),
                dict(), dict(weight=w, gate=d["gate"]), dict(weight=w.cpu()), dict(weight=w, branch=y, eps=0.0),
                dict(weight=w, gate=d["gate"][0], branch=y)):
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            moe.block_norm(x, **bad)
    for bad in (x.t().contiguous().t(), x.double(), x[0], torch.zeros((4, 60), device=dev()), torch.zeros((4, 8200), device=dev())):
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            moe.block_norm(bad, torch.ones(bad.shape[-1], device=dev()))
    _, _, stats = moe.block_norm(x, w, y, save_for_backward=True)
    for args, kw in (((None, up["dr"], x, stats), dict(weight=w, branch=y)), ((up["dh"], up["dr"].float(), x, stats), dict(weight=w, branch=y)),
                     ((up["dh"], up["dr"], x, stats[:1]), dict(weight=w, branch=y)), ((up["dh"], up["dr"], x, None), dict(weight=w, branch=y)),
                     ((up["dh"], up["dr"], x, stats), dict(branch=y)), ((up["dh"][:4], up["dr"], x, stats), dict(weight=w, branch=y))):
        with pytest.raises((ValueError, TypeError)):
            moe.block_norm_bwd(*args, **kw)
