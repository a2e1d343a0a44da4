"""Cases, plain forms and references of the operators around the expert layer.

  few    the whole expert layer for a few tokens: router, choice of experts,
         SwiGLU experts (and the shared one), gate-weighted sum
  norm   a block's norms with its residual: r = a x + b g * rms(branch) v,
         h = rms(r) w
  train  the same, then its gradients for dr and dh
  clip   the 2-norm over a list of gradients, and the gradients scaled to it
  gnorm  the norm alone

``own`` chooses between elementary torch operations in 32 bits (False) and
the framework's calls (True); ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def _few(name, T, H, E, k, I, shared=0, routing=None, bias=False):
    return dict(name=name, op="few", T=T, H=H, E=E, k=k, I=I, shared=shared, bias=bias, routed=routing is not None,
                **(routing or dict(score="softmax", groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0,
                                   balance=False)))


def _norm(name, op, T, H, x, branch=True, post=False, weight=True, gates=0, params="f32", a=1.0, b=1.0):
    return dict(name=name, op=op, T=T, H=H, x=x, branch=branch, post=post, weight=weight, gates=gates, params=params,
                a=a, b=b)


def listed():
    deepseek = dict(score="sigmoid", groups=8, top_groups=4, group_score="top2", renorm=True, scale=2.5, balance=True)
    loose = dict(score="softmax", groups=6, top_groups=3, group_score="max", renorm=False, scale=1.0, balance=False)
    return [
        # one decoded token, Qwen3-MoE shape: latency, eight experts read for one row
        _few("few_qwen_1", 1, 2048, 128, 8, 768),
        # an ordinary decode batch of the same layer
        _few("few_qwen_16", 16, 2048, 128, 8, 768),
        # ragged sizes, groups of experts, weights not renormalised, a bias on the logits
        _few("few_odd_7", 7, 1600, 60, 5, 704, routing=loose, bias=True),
        # the largest: DeepSeek-V3 shape with its shared expert and routing
        _few("few_dsv3_32", 32, 7168, 256, 8, 2048, shared=2048, routing=deepseek),
        # between two blocks of a decoded token, DeepSeek-V3 width: latency
        _norm("norm_1", "norm", 1, 7168, "bf16", params="bf16"),
        # between two blocks of a prefill batch, norms on both sides of the block
        _norm("norm_4096", "norm", 4096, 2048, "bf16", post=True),
        # training micro-batch, residual stream in fp32, a learned scale for each feature
        _norm("train_8191", "train", 8191, 2048, "f32", post=True, gates=1, a=1.0, b=0.5),
        # the largest training batch, a gate for each of 16 sequences, bf16 throughout
        _norm("train_16384", "train", 16384, 7168, "bf16", gates=16, params="bf16"),
        # the gradients of a stack's small parameters (norms, routers' biases): launches
        dict(name="clip_small", op="clip", seed=1, tensors=97, lo=60, hi=16384, types="mixed", total=400000, max_norm=1.0),
        # the gradients of one Qwen3-MoE-shaped layer: gate_up, down, router
        dict(name="clip_layer", op="clip", seed=0, tensors=3, lo=0, hi=0, types="layer", total=604241920, max_norm=1.0),
        # fp32 gradients of odd sizes, the norm that a training loop logs
        dict(name="gnorm_odd", op="gnorm", seed=2, tensors=31, lo=1001, hi=20000001, types="f32", total=60000000,
             max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.random()
    if kind < 0.4:
        while True:
            groups = rng.choice((1, 1, 2, 4, 8, 6))
            E = groups * rng.choice([n for n in (4, 8, 10, 16, 20, 32, 64, 100, 128) if 8 <= n * groups <= 256])
            top = rng.randint(1, groups)
            score = rng.choice(("softmax", "sigmoid"))
            balance = score == "sigmoid" and rng.random() < 0.7
            routing = dict(score=score, groups=groups, top_groups=top,
                           group_score="top2" if balance and groups > 1 and rng.random() < 0.7 else "max",
                           renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), balance=balance)
            I = 64 * _log_int(rng, 4, 46)
            c = _few("", _log_int(rng, 1, 64), 64 * _log_int(rng, 8, 112), E, rng.randint(1, min(8, E // groups * top)), I,
                     shared=rng.choice((0, 0, I, 2 * I)), routing=None if groups == 1 and rng.random() < 0.5 else routing,
                     bias=rng.random() < 0.3)
            if E * c["H"] * I <= 256 * 7168 * 1024:
                break
    elif kind < 0.75:
        while True:
            T, H = _log_int(rng, 1, 16384), 8 * _log_int(rng, 8, 1024)
            divisors = [g for g in range(1, 65) if T % g == 0] + [T]
            branch = rng.random() < 0.85
            c = _norm("", rng.choice(("norm", "train")), T, H, rng.choice(("bf16", "bf16", "f32")), branch=branch,
                      post=branch and rng.random() < 0.5, weight=not branch or rng.random() < 0.8,
                      gates=rng.choice((0, 1, rng.choice(divisors))) if branch else 0, params=rng.choice(("f32", "bf16")),
                      a=rng.choice((1.0, 0.7)) if branch else 1.0, b=rng.choice((1.0, 0.22)) if branch else 1.0)
            if T * H <= 16384 * 4096:
                break
    else:
        n = _log_int(rng, 1, 300)
        lo = _log_int(rng, 1, 5000)
        c = dict(op=rng.choice(("clip", "clip", "gnorm")), seed=rng.randrange(1 << 30), tensors=n, lo=lo,
                 hi=lo * rng.choice((1, 10, 1000)), types=rng.choice(("f32", "bf16", "mixed")),
                 total=_log_int(rng, 1 << 20, 300000000), max_norm=rng.choice((1.0, 0.1, 1e9)))
    c.pop("name", None)
    return c


def _tensors(c):
    """[(elements, dtype)] of a list of gradients, `total` elements at most."""
    if c["types"] == "layer":
        return [(128 * 2048 * 1536, torch.bfloat16), (128 * 768 * 2048, torch.bfloat16), (2048 * 128, torch.float32)]
    import random

    rng = random.Random(c["seed"])
    out, left = [], c["total"]
    for i in range(c["tensors"]):
        n = min(_log_int(rng, c["lo"], max(c["lo"], c["hi"])), max(1, left - (c["tensors"] - 1 - i)))
        left -= n
        t = c["types"] if c["types"] != "mixed" else rng.choice(("f32", "bf16"))
        out.append((n, torch.float32 if t == "f32" else torch.bfloat16))
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def big(rows, cols, scale):
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 27) // cols)
        for r in range(0, rows, step):
            n = min(step, rows - r)
            out[r:r + n] = normal(n, cols) * scale
        return out

    c = dict(case)
    s = dict(case=c)
    if c["op"] == "few":
        T, H, E, I = c["T"], c["H"], c["E"], c["I"]
        s["x"] = normal(T, H).to(torch.bfloat16)
        s["w_router"] = normal(H, E) / math.sqrt(H)
        s["gate_up"], s["down"] = big(E * H, 2 * I, H ** -0.5), big(E * I, H, I ** -0.5)
        n = c["shared"]
        s["sh_gate_up"], s["sh_down"] = (big(H, 2 * n, H ** -0.5), big(n, H, n ** -0.5)) if n else (None, None)
        s["bias"] = 0.2 * normal(E) if c["bias"] else None
        s["balance"] = 0.1 * normal(E) if c["balance"] else None
        return s
    if c["op"] in ("norm", "train"):
        T, H = c["T"], c["H"]
        types = {"f32": torch.float32, "bf16": torch.bfloat16}
        x, p = types[c["x"]], types[c["params"]]
        s["x"] = (3.0 * normal(T, H)).to(x)      # a residual stream has grown over the layers
        s["branch"] = normal(T, H).to(torch.bfloat16) if c["branch"] else None
        s["weight"] = (1.0 + 0.2 * normal(H)).to(p) if c["weight"] else None
        s["post"] = (1.0 + 0.2 * normal(H)).to(p) if c["post"] else None
        s["gate"] = (0.5 * normal(c["gates"], H)).to(p) if c["gates"] else None
        if c["op"] == "train":
            s["dh"] = normal(T, H).to(torch.bfloat16) if c["weight"] else None
            s["dr"] = normal(T, H).to(x) if c["branch"] else None
        return s
    # a training program keeps the gradients of a type in one buffer, whose parts the parameters' gradients are
    sizes = _tensors(c)
    total = sum(n for n, _ in sizes)
    s["grads"], s["flat"], s["out"], s["out_flat"] = [], {}, [], {}
    for t in (torch.float32, torch.bfloat16):
        mine = [(i, n) for i, (n, u) in enumerate(sizes) if u == t]
        if not mine:
            continue
        flat = torch.empty(sum(n for _, n in mine), dtype=t, device=DEV)
        s["flat"][str(t)] = flat
        s["out_flat"][str(t)] = torch.empty_like(flat) if c["op"] == "clip" else flat
        for a, b in ((s["grads"], flat), (s["out"], s["out_flat"][str(t)])):
            a.extend(b.split([n for _, n in mine]))
        for (i, n), part in zip(mine, flat.split([n for _, n in mine])):
            for at in range(0, n, 1 << 27):
                more = part[at:at + (1 << 27)]
                more.copy_(10.0 / math.sqrt(total) * (1 + i % 3) * normal(more.numel()))
    return s


# ------------------------------------------------------------------ plain forms

def _choose(z, c, balance):
    """ids and weights from logits in 64 bits, so that ties are those of the inputs."""
    T, E = z.shape
    groups = c["groups"]
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        s = torch.exp(z - z.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    a = s if balance is None else s + balance
    inside = torch.ones_like(z, dtype=torch.bool)
    if groups > 1:
        by = a.reshape(T, groups, E // groups)
        best = by.amax(2) if c["group_score"] == "max" else by.topk(2, 2).values.sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, groups), dtype=torch.bool, device=z.device).scatter_(1, order[:, :c["top_groups"]], True)
        inside = keep.repeat_interleave(E // groups, 1)
    ids = torch.sort(torch.where(inside, a, -math.inf), dim=1, descending=True, stable=True).indices[:, :c["k"]]
    p = s.gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(1, keepdim=True)
    return ids, c["scale"] * p


def _swiglu(rows, gate_up, down):
    """rows [..., n, H] through weights [..., H, 2I] and [..., I, H] in 32 bits."""
    gu = torch.matmul(rows, gate_up.float())
    g, u = gu.chunk(2, -1)
    return torch.matmul(g / (1.0 + torch.exp(-g)) * u, down.float())


def _plain_few(s):
    c = s["case"]
    T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
    z = torch.matmul(s["x"].double(), s["w_router"].double())
    ids, w = _choose(z if s["bias"] is None else z + s["bias"], c, s["balance"])
    x = s["x"].float()
    gate_up, down = s["gate_up"].view(E, H, 2 * I), s["down"].view(E, I, H)
    if T * k < E:      # the slots' own weights
        e = ids.reshape(-1)
        y = _swiglu(x.repeat_interleave(k, 0).unsqueeze(1), gate_up[e], down[e]).view(T, k, H)
    else:              # every expert on every token, then the slots' own
        every = _swiglu(x, gate_up, down)
        y = every[ids, torch.arange(T, device=x.device).unsqueeze(1)]
    y = (y * w.float().unsqueeze(2)).sum(1)
    if s["sh_gate_up"] is not None:
        y = y + _swiglu(x, s["sh_gate_up"], s["sh_down"])
    return dict(y=y.to(torch.bfloat16), ids=ids.to(torch.int32), w=w.float())


def _rms(v):
    return 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    T, H, groups = c["T"], c["H"], max(1, c["gates"])
    x = s["x"].float()
    w = None if s["weight"] is None else s["weight"].float()
    out = {}
    r, sy, y, n, gate = x, None, None, None, None
    if s["branch"] is not None:
        y = s["branch"].float()
        n = y
        if s["post"] is not None:
            sy = _rms(y)
            n = y * sy * s["post"].float()
        z = n
        if s["gate"] is not None:
            gate = s["gate"].float().repeat_interleave(T // groups, 0)
            z = n * gate
        r = c["a"] * x + c["b"] * z
        out["r"] = r.to(s["x"].dtype)
    if w is not None:
        sr = _rms(r)
        out["h"] = (r * sr * w).to(torch.bfloat16)
    if c["op"] == "norm":
        return out
    d = torch.zeros_like(x) if s["dr"] is None else s["dr"].float()
    if w is not None:
        dh, xn = s["dh"].float(), r * sr
        t = dh * w
        d = d + sr * (t - xn * (t * xn).mean(1, keepdim=True))
        out["d_weight"] = (dh * xn).sum(0).to(s["weight"].dtype)
    out["dx"] = (c["a"] * d).to(s["x"].dtype)
    if y is not None:
        dn = c["b"] * d
        if gate is not None:
            out["d_gate"] = (dn * n).view(groups, T // groups, H).sum(1).to(s["gate"].dtype)
            dn = dn * gate
        if sy is not None:
            yn = y * sy
            out["d_post"] = (dn * yn).sum(0).to(s["post"].dtype)
            t = dn * s["post"].float()
            dn = sy * (t - yn * (t * yn).mean(1, keepdim=True))
        out["d_branch"] = dn.to(torch.bfloat16)
    return out


def _plain_clip(s):
    grads = [g.float() for g in s["grads"]]
    norm = torch.stack([g.square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()
    if s["case"]["op"] == "gnorm":
        return dict(norm=norm)
    scale = torch.clamp(s["case"]["max_norm"] / (norm + EPS), max=1.0)
    for o, g in zip(s["out"], grads):
        o.copy_(g * scale)
    return dict(norm=norm, grads=s["out_flat"])


def _own(s):
    import token_dispatch_grouped_softmax_gb300 as moe

    c = s["case"]
    if c["op"] == "few":
        routing = None
        if c["routed"]:
            routing = moe.Routing(score=c["score"], n_groups=c["groups"], top_groups=c["top_groups"],
                                  group_score=c["group_score"], renorm=c["renorm"], scale=c["scale"])
        y, ids, w = moe.moe_forward_few(s["x"], s["w_router"], s["gate_up"], s["down"], c["k"], bias=s["bias"],
                                        sh_gate_up=s["sh_gate_up"], sh_down=s["sh_down"], routing=routing,
                                        balance_bias=s["balance"])
        return dict(y=y, ids=ids, w=w)
    if c["op"] in ("norm", "train"):
        how = dict(weight=s["weight"], branch=s["branch"], post_weight=s["post"], gate=s["gate"], residual_scale=c["a"],
                   branch_scale=c["b"])
        r, h, stats = moe.block_norm(s["x"], eps=EPS, save_for_backward=c["op"] == "train", **how)
        out = {}
        if r is not None:
            out["r"] = r
        if h is not None:
            out["h"] = h
        if c["op"] == "train":
            grads = moe.block_norm_bwd(s["dh"], s["dr"], s["x"], stats, **how)
            for name, mine in (("d_weight", "d_weight"), ("dx", "dx"), ("d_gate", "d_gate"), ("d_post", "d_post_weight"),
                               ("d_branch", "d_branch")):
                if grads[mine] is not None:
                    out[name] = grads[mine]
        return out
    if c["op"] == "gnorm":
        return dict(norm=moe.grad_norm(s["grads"]))
    return dict(norm=moe.clip_grads(s["grads"], c["max_norm"], out=s["out"]), grads=s["out_flat"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_few(state) if op == "few" else _plain_norm(state) if op in ("norm", "train") else _plain_clip(state)


# ------------------------------------------------------------------- what it is

def work(case):
    c = case
    if c["op"] == "few":
        T, H, E, k, I, n = c["T"], c["H"], c["E"], c["k"], c["I"], c["shared"]
        used = E * (1.0 - (1.0 - k / E) ** T)     # distinct experts of T tokens, each choosing k of E evenly
        b = used * 6 * H * I + 6 * H * n + 4 * H * E + 4 * T * H + 8 * T * k
        return dict(bytes=b, flops=2.0 * T * (H * E + 3 * H * (k * I + n)))
    if c["op"] in ("norm", "train"):
        T, H = c["T"], c["H"]
        xs, ps = (4 if c["x"] == "f32" else 2), (4 if c["params"] == "f32" else 2)
        params = (c["weight"] + c["post"] + c["gates"]) * H * ps
        b = T * H * (xs + (2 + xs) * c["branch"] + 2 * c["weight"]) + params
        f = 12 * T * H
        if c["op"] == "train":    # x and branch are read by both directions
            b += T * H * (2 * xs + (4 + xs) * c["branch"] + 2 * c["weight"]) + 2 * params
            f += 24 * T * H
        return dict(bytes=b, flops=f)
    sizes = [(n, 2 if t == torch.bfloat16 else 4) for n, t in _tensors(c)]
    total = sum(n for n, _ in sizes)
    b = sum(n * e for n, e in sizes)
    return dict(bytes=b + 4 if c["op"] == "gnorm" else 2 * b + 4, flops=2 * total if c["op"] == "gnorm" else 3 * total)


def _exact_few(s):
    c = s["case"]
    T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
    x = s["x"].double()
    z = torch.einsum("th,he->te", x, s["w_router"].double())
    if s["bias"] is not None:
        z = z + s["bias"].double()
    score = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    value = score if s["balance"] is None else score + s["balance"].double()
    per = E // c["groups"]
    table = value.reshape(T, c["groups"], per).sort(dim=2, descending=True).values
    strength = table[:, :, 0] if c["group_score"] == "max" or per == 1 else table[:, :, :2].sum(2)
    rank = torch.argsort(torch.argsort(strength, dim=1, descending=True, stable=True), 1)
    outside = (rank >= c["top_groups"]).unsqueeze(2).expand(T, c["groups"], per).reshape(T, E)
    ids = value.masked_fill(outside, -1e300).argsort(dim=1, descending=True, stable=True)[:, :k]
    chosen = score.gather(1, ids)
    w = c["scale"] * (chosen / chosen.sum(1, keepdim=True) if c["renorm"] else chosen)
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)

    def expert(rows, gate_up, down):
        g, u = (rows @ gate_up.double()).split(down.shape[0], 1)
        return (torch.nn.functional.silu(g) * u) @ down.double()

    for e in sorted(set(ids.reshape(-1).tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        y[t] += w[t, j].unsqueeze(1) * expert(x[t], s["gate_up"][e * H:(e + 1) * H], s["down"][e * I:(e + 1) * I])
    if s["sh_gate_up"] is not None:
        y += expert(x, s["sh_gate_up"], s["sh_down"])
    return dict(y=y, ids=ids.to(torch.int32), w=w)


def _exact_norm(s):
    c = s["case"]
    leaves = {n: None if s[n] is None else s[n].double().requires_grad_(c["op"] == "train")
              for n in ("x", "branch", "weight", "post", "gate")}

    def rms_norm(v, weight):
        return v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).pow(0.5) * weight

    out = {}
    r = leaves["x"]
    if c["branch"]:
        z = leaves["branch"] if leaves["post"] is None else rms_norm(leaves["branch"], leaves["post"])
        if leaves["gate"] is not None:
            z = (z.view(c["gates"], -1, c["H"]) * leaves["gate"].unsqueeze(1)).view(c["T"], c["H"])
        r = c["a"] * r + c["b"] * z
        out["r"] = r
    if c["weight"]:
        out["h"] = rms_norm(r, leaves["weight"])
    if c["op"] == "train":
        pairs = [(out[o], s[d].double()) for o, d in (("h", "dh"), ("r", "dr")) if o in out]
        torch.autograd.backward([o for o, _ in pairs], [d for _, d in pairs])
        out = {n: v.detach() for n, v in out.items()}
        for name, leaf in (("d_weight", "weight"), ("dx", "x"), ("d_gate", "gate"), ("d_post", "post"), ("d_branch", "branch")):
            if leaves[leaf] is not None:
                out[name] = leaves[leaf].grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        if case["op"] == "few":
            return _exact_few(s)
        if case["op"] in ("norm", "train"):
            return _exact_norm(s)
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
    answer = dict(norm=torch.tensor(norm, dtype=torch.float64, device=DEV))
    if case["op"] == "clip":
        answer["grads"] = {t: g.double() * min(1.0, case["max_norm"] / (norm + EPS)) for t, g in s["flat"].items()}
    return answer
