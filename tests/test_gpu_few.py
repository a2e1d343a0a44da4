"""The expert layer for a few tokens against the formula in 64 bits.

Tolerances, from the arithmetic, all in terms of the formula with positive
terms: u = 2^-24.  A sum over K in fp32 is off by at most K u of the sum of
its terms' sizes; silu and the product with u add 2^-20 of h; h is rounded
to bf16 (half a step, 2^-8 of it); y to bf16."""
import pytest
import torch

from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu


def weights(E, H, I, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    bf = lambda *s, scale: (scale * torch.randn(s, generator=g, device=dev())).to(torch.bfloat16)
    return bf(E * H, 2 * I, scale=H ** -0.5), bf(E * I, H, scale=I ** -0.5)


def make(T, H, E, k, I, I_s=0, seed=0, distinct=True):
    g = torch.Generator(device=dev()).manual_seed(seed + 77)
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    if distinct:
        ids = torch.rand((T, E), generator=g, device=dev()).argsort(1)[:, :k].to(torch.int32).contiguous()
    else:
        ids = torch.randint(0, E, (T, k), generator=g, device=dev(), dtype=torch.int32)
    w = torch.randn((T, k), generator=g, device=dev()).softmax(1)
    gu, dn = weights(E, H, I, seed)
    sh = weights(1, H, I_s, seed + 1) if I_s else (None, None)
    return x, ids, w, gu, dn, sh[0], sh[1]


def reference(x, ids, w, gate_up, down, sh_gate_up=None, sh_down=None):
    """y in 64 bits and how far an output may be off."""
    T, H = x.shape
    E = gate_up.shape[0] // H
    I = down.shape[0] // E
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    allow = torch.zeros_like(y)
    u32 = 2.0 ** -24

    def expert(rows, wt, gu, dn):
        I = dn.shape[0]
        gu, dn = gu.double(), dn.double()
        z, a = rows @ gu, rows.abs() @ gu.abs()
        ez = rows.shape[1] * u32 * a
        g, u = z[:, :I], z[:, I:]
        s = g * torch.sigmoid(g)
        h = s * u
        eh = 1.1 * ez[:, :I] * (u.abs() + ez[:, I:]) + s.abs() * ez[:, I:] + 2.0 ** -20 * h.abs()
        eh = eh + (h.abs() + eh) * 2.0 ** -8
        big = (h.abs() + eh) @ dn.abs()
        return wt * (h @ dn), wt.abs() * (eh @ dn.abs() + (I + 40) * u32 * big)

    def add(t, part):
        y.index_add_(0, t, part[0])
        allow.index_add_(0, t, part[1])

    for e in sorted(set(ids.reshape(-1).tolist())):
        if 0 <= e < E:
            t, j = (ids == e).nonzero(as_tuple=True)
            add(t, expert(x[t].double(), w[t, j].double().unsqueeze(1), gate_up[e * H:(e + 1) * H], down[e * I:(e + 1) * I]))
    if sh_gate_up is not None:
        t = torch.arange(T, device=x.device)
        add(t, expert(x.double(), torch.ones((T, 1), dtype=torch.float64, device=x.device), sh_gate_up, sh_down))
    return y, allow + 2.0 ** -8 * (y.abs() + allow)


def close(y, want):
    ref, allow = want
    err = (y.double() - ref).abs()
    assert bool(torch.isfinite(y).all()) and bool((err <= allow).all()), float((err - allow).max())
    # and the sum over an output's row as a whole: rounding errors are not all of one sign
    rel = float(err.norm() / ref.norm()) if float(ref.norm()) > 0 else 0.0
    assert rel < 2.0 ** -7, rel


SHAPES = [(1, 64, 1, 1, 64, 0), (2, 1024, 4, 1, 64, 3200), (70, 1024, 4, 1, 64, 3200), (40, 512, 40, 4, 1024, 64), (1, 128, 8, 2, 64, 0), (1, 2048, 128, 8, 768, 0), (3, 192, 5, 3, 320, 64), (2, 1600, 60, 5, 704, 0),
          (16, 2048, 32, 8, 768, 768), (64, 256, 16, 8, 128, 192), (128, 128, 8, 8, 64, 64), (37, 1088, 24, 6, 448, 896), (5, 7168, 16, 8, 2048, 2048),
          (33, 64, 64, 32, 64, 64), (9, 4096, 8, 2, 64, 0), (4, 64, 4, 1, 8192, 0), (128, 320, 3, 1, 192, 0), (31, 512, 1024, 32, 64, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_experts(shape):
    moe = lib()
    T, H, E, k, I, I_s = shape
    a = make(T, H, E, k, I, I_s)
    y = moe.experts_few(*a)
    moe.sync_status()
    close(y, reference(*a))


def test_every_token_to_one_expert_and_the_same_expert_twice():
    moe = lib()
    T, H, E, k, I = 128, 256, 8, 8, 192
    x, ids, w, gu, dn, _, _ = make(T, H, E, k, I, distinct=False)
    close(moe.experts_few(x, ids, w, gu, dn), reference(x, ids, w, gu, dn))
    ids.fill_(5)                                            # 1024 rows of one expert
    close(moe.experts_few(x, ids, w, gu, dn), reference(x, ids, w, gu, dn))
    moe.sync_status()


@pytest.mark.parametrize("shared", (0, 128))
def test_empty_slots(shared):
    """Padded tokens and single empty slots; what their w holds does not count."""
    moe = lib()
    T, H, E, k, I = 21, 256, 16, 4, 128
    a = list(make(T, H, E, k, I, shared))
    a[1][15:] = -1
    a[1][3, 2] = -1
    a[1][4] = -1
    want = reference(*a)
    a[2][15:] = float("nan")
    a[2][3, 2] = float("inf")
    y = moe.experts_few(*a)
    moe.sync_status()
    close(y, want)
    if not shared:
        assert bool((y[15:] == 0).all()) and bool((y[4] == 0).all())
    a[1].fill_(-1)
    y = moe.experts_few(*a)
    close(y, reference(*a))


def test_bad_ids_are_reported_and_empty():
    moe = lib()
    a = list(make(6, 128, 8, 2, 64))
    a[1][2, 1] = 8
    a[1][4, 0] = -7
    y = moe.experts_few(*a)
    with pytest.raises(moe.MoEError, match="MOE_ERR_DEVICE"):
        moe.sync_status()
    close(y, reference(*a))
    moe.sync_status()


@pytest.mark.parametrize("shape", [(64, 512, 32, 8, 256, 192), (128, 1024, 8, 2, 704, 0)], ids=str)
def test_a_token_does_not_depend_on_the_batch(shape):
    moe = lib()
    T, H, E, k, I, I_s = shape
    x, ids, w, gu, dn, sgu, sdn = make(T, H, E, k, I, I_s)
    y = moe.experts_few(x, ids, w, gu, dn, sgu, sdn)
    for a, b in ((0, 1), (5, 12), (20, 60), (T - 1, T)):
        part = moe.experts_few(x[a:b], ids[a:b].contiguous(), w[a:b].contiguous(), gu, dn, sgu, sdn)
        assert torch.equal(part, y[a:b])
    moe.sync_status()


def test_infinities_and_nan_stay_in_their_tokens():
    moe = lib()
    x, ids, w, gu, dn, sgu, sdn = make(30, 256, 8, 3, 128, 64)
    clean = moe.experts_few(x, ids, w, gu, dn, sgu, sdn)
    x[7, 3] = float("inf")
    x[20, 200] = float("nan")
    y = moe.experts_few(x, ids, w, gu, dn, sgu, sdn)
    ok = [t for t in range(30) if t not in (7, 20)]
    assert torch.equal(y[ok], clean[ok]) and bool(y[20].isnan().all()) and not bool(y[7].isfinite().all())
    # a weight of an expert that no token has may hold anything
    used = set(ids.reshape(-1).tolist())
    x, ids, w, gu, dn, _, _ = make(3, 256, 64, 3, 128)
    free = [e for e in range(64) if e not in set(ids.reshape(-1).tolist())]
    clean = moe.experts_few(x, ids, w, gu, dn)
    for e in free:
        gu[e * 256:(e + 1) * 256] = float("nan")
        dn[e * 128:(e + 1) * 128] = float("nan")
    assert used and torch.equal(moe.experts_few(x, ids, w, gu, dn), clean)
    moe.sync_status()


def test_no_tokens():
    moe = lib()
    x, ids, w, gu, dn, _, _ = make(1, 128, 8, 2, 64)
    y = moe.experts_few(x[:0], ids[:0], w[:0], gu, dn)
    assert y.shape == (0, 128)
    y, i, q = moe.layer_few(x[:0], torch.zeros((128, 8), device=dev()), gu, dn, 2)
    assert y.shape == (0, 128) and i.shape == q.shape == (0, 2)


def test_out():
    """out: a row slice, its neighbours untouched."""
    moe = lib()
    a = make(5, 128, 8, 2, 64)
    buffer = torch.full((9, 128), 5.0, dtype=torch.bfloat16, device=dev())
    y = moe.experts_few(*a, out=buffer[2:7])
    assert y.data_ptr() == buffer[2:7].data_ptr() and torch.equal(buffer[2:7], moe.experts_few(*a))
    assert bool((buffer[:2] == 5).all()) and bool((buffer[7:] == 5).all())


@pytest.mark.parametrize("T", (1, 7, 64, 128))
@pytest.mark.parametrize("kw", (None, dict(score="sigmoid", n_groups=4, top_groups=2, scale=2.5), dict(renorm=False), dict(score="sigmoid", renorm=False),
                                dict(n_groups=4, top_groups=3, group_score="max")), ids=str)
def test_layer(T, kw):
    """The whole layer: the choice that route_select makes of the logits in 64
    bits where no two of them nearly tie, its weights, and the experts'
    output, with a bias on the logits and one on the choice."""
    moe = lib()
    H, E, k, I, I_s = 320, 64, 4, 128, 64
    x, _, _, gu, dn, sgu, sdn = make(T, H, E, k, I, I_s, seed=T)
    g = torch.Generator(device=dev()).manual_seed(T)
    wr = torch.randn((H, E), generator=g, device=dev()) * H ** -0.5
    bias = 0.3 * torch.randn(E, generator=g, device=dev())
    routing = None if kw is None else moe.Routing(**kw)
    how = moe.Routing() if kw is None else routing
    balance = 0.1 * torch.randn(E, generator=g, device=dev()) if kw and kw.get("score") == "sigmoid" else None
    y, ids, w = moe.moe_forward_few(x, wr, gu, dn, k, bias=bias, sh_gate_up=sgu, sh_down=sdn, routing=routing, balance_bias=balance)
    moe.sync_status()
    z = x.double() @ wr.double() + bias.double()
    size = x.double().abs() @ wr.double().abs() + bias.double().abs()
    near = float((size * (H + 16) * 2.0 ** -24).max())       # how far an fp32 logit may be off
    want, _ = how.select(z.float().contiguous(), k, balance)
    assert torch.equal(ids, want)      # the seeds' logits have no near ties
    s = torch.sigmoid(z) if how.score == "sigmoid" else torch.softmax(z, 1)
    p = s.gather(1, ids.long())
    p = how.scale * (p / p.sum(1, keepdim=True) if how.renorm else p)
    assert bool(((w.double() - p).abs() <= (4 * near + 2.0 ** -20) * p).all())
    close(y, reference(x, ids, w, gu, dn, sgu, sdn))


@pytest.mark.parametrize("E", (1, 2, 3, 33, 255, 256, 260, 511, 513, 1000, 1021, 1024))
@pytest.mark.parametrize("T", (1, 3, 9))
def test_layer_any_number_of_experts(E, T):
    """The router's ids and weights for every layout of its columns, with the experts' own weights small."""
    moe = lib()
    H, I, k = 64 * (1 + E % 3), 64, min(E, 1 + E % 5)
    g = torch.Generator(device=dev()).manual_seed(E)
    x = torch.randn((T, H), generator=g, device=dev()).to(torch.bfloat16)
    gu, dn = weights(E, H, I, E)
    # logits a step of 2^-8 apart at least: no near ties
    wr = torch.zeros((H, E), device=dev())
    x[:, 0] = 1.0
    wr[0] = torch.randperm(E, generator=g, device=dev()) * 2.0 ** -7
    wr[1:] = 2.0 ** -14 * torch.randn((H - 1, E), generator=g, device=dev()) / H ** 0.5
    y, ids, w = moe.layer_few(x, wr, gu, dn, k)
    z = x.double() @ wr.double()
    want = z.sort(1, descending=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    p = torch.softmax(z.gather(1, want), 1)
    assert bool(((w.double() - p).abs() <= 2.0 ** -18 * p).all())
    close(y, reference(x, ids, w, gu, dn))


def test_layer_masked_and_tied_experts():
    """Logits of -inf (masked by the bias), and equal ones, which go to the lower index."""
    moe = lib()
    x, _, _, gu, dn, _, _ = make(5, 128, 8, 4, 64)
    wr = torch.zeros((128, 8), device=dev())
    bias = torch.tensor([0.0, -float("inf"), 0.0, 0.0, -float("inf"), 0.0, 0.0, 0.0], device=dev())
    y, ids, w = moe.moe_forward_few(x, wr, gu, dn, 4, bias=bias)
    assert ids.tolist() == [[0, 2, 3, 5]] * 5 and bool((w == 0.25).all())
    close(y, reference(x, ids, w, gu, dn))
    y, ids, w = moe.moe_forward_few(x, wr, gu, dn, 8, bias=bias)     # masked ones last, with weight 0
    assert bool((w[:, 6:] == 0).all()) and set(ids[0, 6:].tolist()) == {1, 4}
    close(y, reference(x, ids, w, gu, dn))
    bias.fill_(-float("inf"))
    y, ids, w = moe.moe_forward_few(x, wr, gu, dn, 4, bias=bias)     # nothing is left
    assert bool((w == 0).all()) and bool((y == 0).all())
    moe.sync_status()


def test_layer_equals_its_steps():
    moe = lib()
    x, _, _, gu, dn, sgu, sdn = make(12, 256, 16, 4, 128, 64)
    wr = torch.randn((256, 16), generator=torch.Generator().manual_seed(1)).to(dev()) / 16
    y, ids, w = moe.layer_few(x, wr, gu, dn, 4, sh_gate_up=sgu, sh_down=sdn)
    assert torch.equal(y, moe.experts_few(x, ids, w, gu, dn, sgu, sdn))
    for a, b in ((0, 1), (3, 9)):
        yp, ip, wp = moe.layer_few(x[a:b], wr, gu, dn, 4, sh_gate_up=sgu, sh_down=sdn)
        assert torch.equal(yp, y[a:b]) and torch.equal(ip, ids[a:b]) and torch.equal(wp, w[a:b])


def test_two_streams_and_graphs():
    """Calls at the same time on two streams, and two captured graphs replayed
    in turn and together, with inputs that change."""
    moe = lib()
    a, b = make(16, 512, 16, 4, 256, 128, seed=1), make(40, 512, 16, 4, 256, 0, seed=2)
    want = [moe.experts_few(*a), moe.experts_few(*b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.experts_few(*(a, b)[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    wr = torch.randn((512, 16), generator=torch.Generator().manual_seed(1)).to(dev()) / 16
    graphs, outs = [], []
    for i, c in enumerate((a, b)):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(moe.layer_few(c[0], wr, c[3], c[4], 4, sh_gate_up=c[5], sh_down=c[6]))
        graphs.append(g)
    for step in range(3):
        for c in (a, b):
            c[0].add_(0.25)
        want = [moe.layer_few(c[0], wr, c[3], c[4], 4, sh_gate_up=c[5], sh_down=c[6]) for c in (a, b)]
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for o, t in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, t))
    moe.sync_status()


def test_refusals():
    moe = lib()
    x, ids, w, gu, dn, sgu, sdn = make(4, 128, 8, 2, 64, 64)
    for bad in ((x.float(), ids, w, gu, dn), (x, ids.long(), w, gu, dn), (x, ids[:2], w, gu, dn), (x, ids, w[:, :1], gu, dn), (x, ids, w, gu[:100], dn),
                (x, ids, w, gu, dn[:, :64]), (x, ids, w, gu, dn[:64]), (x, ids, w, gu, dn, sgu), (x, ids, w, gu, dn, None, sdn), (x, ids, w, gu, dn, sgu[:64], sdn),
                (x, ids, w, gu, dn, sgu, sdn[:32]), (x.cpu(), ids, w, gu, dn), (x, ids, w, gu, dn, None, None, torch.empty_like(x)[:2]),
                (x, ids, w.t().contiguous().t(), gu, dn)):
        with pytest.raises((ValueError, TypeError)):
            moe.experts_few(*bad)
    big = torch.zeros((129, 128), dtype=torch.bfloat16, device=dev())
    with pytest.raises(moe.MoEError):
        moe.experts_few(big, torch.zeros((129, 1), dtype=torch.int32, device=dev()), torch.ones((129, 1), device=dev()), gu, dn)
    wr = torch.zeros((128, 8), device=dev())
    for kw in (dict(k=9), dict(k=0), dict(k=2, n_groups=3), dict(k=2, score="relu"), dict(k=2, scale=float("nan")), dict(k=2, bias=wr[0, :4])):
        k = kw.pop("k")
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            moe.layer_few(x, wr, gu, dn, k, **kw)
    with pytest.raises(ValueError):
        moe.layer_few(x, wr[:, :4].contiguous(), gu, dn, 2)
    with pytest.raises(ValueError):
        moe.moe_forward_few(x, wr, gu, dn, 2, balance_bias=wr[0])
