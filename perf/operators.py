"""Cases, plain forms and references of the expert-choice and 4-bit expert operators.

  route     logits -> scores, groups, top-k ids and weights
  train     the same, then its gradient and the balance bias's update
  gate_up   4-bit experts of a decode batch: h = silu(x.Wg) * (x.Wu)
  down      4-bit experts of a decode batch: y = sum_j w_j h_j.Wd

``own`` chooses between elementary torch operations in 32 bits (False) and
the framework's calls (True); ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decoded token through the DeepSeek-V3-shaped router: latency alone
        dict(name="route_decode_1", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_score="top2", renorm=True, scale=2.5, dtype="f32"),
        # a prefill chunk of the Qwen3-MoE-shaped layer (softmax, one group)
        dict(name="route_softmax_4096", op="route", T=4096, E=128, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renorm=True, scale=1.0, dtype="f32"),
        # the DeepSeek-V3-shaped prefill batch
        dict(name="route_sigmoid_16384", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, dtype="f32"),
        # ragged batch, odd expert counts, bf16 logits, groups chosen by their best expert
        dict(name="route_odd_1021", op="route", T=1021, E=60, k=5, score="softmax", bias=False, groups=6,
             top_groups=3, group_score="max", renorm=False, scale=1.0, dtype="bf16"),
        # training micro-batch, sigmoid scores with the balance bias and its update
        dict(name="train_sigmoid_8192", op="train", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, dtype="f32"),
        # training micro-batch, softmax weights that are not renormalised: a dense gradient, bf16 logits
        dict(name="train_softmax_8191", op="train", T=8191, E=128, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renorm=False, scale=1.0, dtype="bf16"),
        # one decoded token, Qwen3-MoE shape: eight experts are read for one row
        dict(name="gate_up_qwen_1", op="gate_up", T=1, H=2048, E=128, k=8, I=768, group=128, zeros=False, pad=False),
        # an ordinary decode batch with zero points and some empty (padded) slots, ragged rows per expert
        dict(name="gate_up_qwen_45", op="gate_up", T=45, H=2048, E=128, k=8, I=768, group=64, zeros=True, pad=True),
        # the largest: DeepSeek-V3 shape, most experts in use
        dict(name="gate_up_dsv3_32", op="gate_up", T=32, H=7168, E=256, k=8, I=2048, group=128, zeros=False, pad=False),
        # one decoded token through down and combine
        dict(name="down_qwen_1", op="down", T=1, H=2048, E=128, k=8, I=768, group=128, zeros=False, pad=False),
        # an ordinary decode batch, zero points, empty slots
        dict(name="down_qwen_45", op="down", T=45, H=2048, E=128, k=8, I=768, group=64, zeros=True, pad=True),
        # DeepSeek-V3 shape, most experts in use
        dict(name="down_dsv3_32", op="down", T=32, H=7168, E=256, k=8, I=2048, group=128, zeros=False, pad=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        op = rng.choice(("route", "train"))
        groups = rng.choice((1, 1, 2, 4, 8, 3, 6))
        E = groups * rng.choice([n for n in (4, 8, 10, 16, 20, 32, 64, 100, 128) if 8 <= n * groups <= 256])
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * top_groups))
        score = rng.choice(("softmax", "sigmoid"))
        bias = score == "sigmoid" and rng.random() < 0.7
        T = _log_int(rng, 1, 16384 if op == "route" else 8192)
        if 3072 in (T, T * k):
            T += 1
        return dict(op=op, T=T, E=E, k=k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                    group_score="top2" if bias and groups > 1 and rng.random() < 0.7 else "max",
                    renorm=k > 1 and rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), dtype=rng.choice(("f32", "f32", "bf16")))
    while True:
        op = rng.choice(("gate_up", "down"))
        group = rng.choice((32, 64, 128))
        step = max(64, group)
        c = dict(op=op, T=_log_int(rng, 1, 64), H=step * _log_int(rng, 512 // step, 7168 // step),
                 E=rng.choice((8, 32, 60, 64, 128, 160, 256)), k=rng.randint(1, 8),
                 I=step * _log_int(rng, 256 // step, 2944 // step), group=group, zeros=rng.random() < 0.4,
                 pad=rng.random() < 0.3)
        c["pad"] = c["pad"] and c["T"] > 1
        sizes = (c["H"], c["I"], 2 * c["I"], c["T"] * c["k"])
        weights = c["E"] * c["H"] * c["I"]
        if 3072 not in sizes and weights <= 256 * 7168 * 512:
            return c


def _cols(case):
    """(K, N) of one expert's weight."""
    return (case["H"], 2 * case["I"]) if case["op"] == "gate_up" else (case["I"], case["H"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    c = dict(case)
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] in ("route", "train"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s = dict(case=c, logits=normal(T, E).to(dt).contiguous(), bias=0.1 * normal(E) if c["bias"] else None)
        if c["op"] == "train":
            s["dw"] = normal(T, k)
            # loads of the step before, as the permutation counted them
            load = torch.randint(0, E, (T * k,), generator=g, device=DEV)
            s["counts"] = torch.zeros(E, dtype=torch.int32, device=DEV).index_add_(
                0, load, torch.ones(T * k, dtype=torch.int32, device=DEV))
        return s
    K, N = _cols(c)
    G = c["group"]
    q = torch.empty((E * K // 8, N), dtype=torch.int32, device=DEV)
    rows = max(1, (1 << 24) // N)
    for r0 in range(0, q.shape[0], rows):   # codes of normal weights, about 3.2 steps to a deviation
        r1 = min(q.shape[0], r0 + rows)
        codes = (3.2 * normal(r1 - r0, 8, N) + 8.0).round_().clamp_(0, 15).to(torch.int32)
        word = codes[:, 0].clone()
        for i in range(1, 8):
            word |= codes[:, i] << (4 * i)
        q[r0:r1] = word
    scales = ((0.75 + 0.5 * torch.rand((E * K // G, N), generator=g, device=DEV)) / (3.2 * math.sqrt(K))).to(torch.bfloat16)
    zeros = torch.randint(5, 12, (E * K // G, N), generator=g, device=DEV).to(torch.uint8) if c["zeros"] else None
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    if c["pad"]:   # the batch's last tokens are padding: their slots name no expert
        ids[T - max(1, T // 8):] = -1
    s = dict(case=c, ids=ids, q=q, scales=scales, zeros=zeros)
    if c["op"] == "gate_up":
        s["x"] = normal(T, K).to(torch.bfloat16)
    else:
        s["h"] = (0.6 * normal(T, k, K) * normal(T, k, K).sigmoid()).to(torch.bfloat16)
        s["w"] = normal(T, k).softmax(1).contiguous()
    return s


# ------------------------------------------------------------------ plain forms

def _choose(z, c, bias):
    """ids and weights from fp32 logits."""
    T, E = z.shape
    k, groups = c["k"], c["groups"]
    masked = z == -math.inf
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        s = torch.exp(z - z.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    if bias is None and (groups == 1 or c["group_score"] == "max"):
        a = z
    else:
        a = s if bias is None else s + bias
        a = torch.where(masked, -math.inf, a)
    inside = torch.ones_like(masked)
    if groups > 1:
        by = a.view(T, groups, E // groups)
        if c["group_score"] == "max" or E == groups:
            best = by.amax(2)
        else:
            two = by.topk(2, 2).values
            best = two[:, :, 0] + torch.where(two[:, :, 1] == -math.inf, 0.0, two[:, :, 1])
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, groups), dtype=torch.bool, device=z.device).scatter_(1, order[:, :c["top_groups"]], True)
        inside = keep.repeat_interleave(E // groups, 1)
    first = torch.sort(a, dim=1, descending=True, stable=True).indices
    ids = first.gather(1, torch.sort(inside.gather(1, first).to(torch.uint8), dim=1, descending=True, stable=True).indices[:, :k])
    p = s.gather(1, ids)
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return ids, c["scale"] * p, s


def _choose_bwd(z, c, ids, s, dw):
    p = s.gather(1, ids)
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        u = torch.where(total > 0, p / total, 0.0)
        dq = dw - (u * dw).sum(1, keepdim=True)
        if c["score"] == "softmax":
            d = c["scale"] * u * dq
        else:
            d = c["scale"] * u * dq / (1.0 + torch.exp(z.gather(1, ids)))
        return torch.zeros_like(z).scatter_(1, ids, d)
    if c["score"] == "sigmoid":
        return torch.zeros_like(z).scatter_(1, ids, c["scale"] * dw * p / (1.0 + torch.exp(z.gather(1, ids))))
    back = torch.zeros_like(z).scatter_(1, ids, dw)
    return c["scale"] * s * (back - (p * dw).sum(1, keepdim=True))


def _unpack(q, scales, zeros, K, N, group):
    """[n, K/8, N] words, [n, K/group, N] scales -> [n, K, N] fp32 weights."""
    n = q.shape[0]
    shift = torch.arange(0, 32, 4, dtype=torch.int32, device=q.device).view(1, 1, 8, 1)
    v = ((q.unsqueeze(2) >> shift) & 15).float().view(n, K // group, group, N)
    v = v - (8.0 if zeros is None else zeros.float().unsqueeze(2))
    return (v * scales.float().unsqueeze(2)).view(n, K, N)


def _experts(s, rows, T, k):
    """rows [T, k, K] fp32 through each slot's expert: [T, k, N] fp32, empty slots 0."""
    c = s["case"]
    K, N = _cols(c)
    E, G = c["E"], c["group"]
    q, sc = s["q"].view(E, K // 8, N), s["scales"].view(E, K // G, N)
    zp = None if s["zeros"] is None else s["zeros"].view(E, K // G, N)
    used = s["ids"] >= 0
    e = s["ids"].clamp(min=0).long().view(-1)
    if T * k < E:      # the slots' own weights
        w = _unpack(q[e], sc[e], None if zp is None else zp[e], K, N, G)
        out = torch.bmm(rows.reshape(T * k, 1, K), w).view(T, k, N)
    elif c["op"] == "gate_up":   # every expert on every token, then the slots' own
        w = _unpack(q, sc, zp, K, N, G)
        every = torch.matmul(rows[:, 0], w)                         # [E, T, N]
        at = torch.arange(T, device=e.device).repeat_interleave(k)
        out = every[e, at].view(T, k, N)
    else:
        w = _unpack(q, sc, zp, K, N, G)
        every = torch.matmul(rows.reshape(T * k, K), w)             # [E, T*k, N]
        out = every[e, torch.arange(T * k, device=e.device)].view(T, k, N)
    return torch.where(used.unsqueeze(2), out, 0.0)


def _plain(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    if c["op"] in ("route", "train"):
        z = s["logits"].float()
        ids, w, score = _choose(z, c, s["bias"])
        if c["op"] == "route":
            return dict(ids=ids.to(torch.int32), w=w)
        out = dict(ids=ids.to(torch.int32), w=w, d_logits=_choose_bwd(z, c, ids, score, s["dw"]).to(s["logits"].dtype))
        if s["bias"] is not None:
            n = s["counts"]
            out["bias"] = s["bias"] + 0.001 * torch.sign(n.sum() - c["E"] * n.long()).float()
        return out
    if c["op"] == "gate_up":
        gu = _experts(s, s["x"].float().unsqueeze(1).expand(T, k, c["H"]), T, k)
        g, u = gu[..., :c["I"]], gu[..., c["I"]:]
        return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
    y = _experts(s, s["h"].float(), T, k)
    return (y * s["w"].unsqueeze(2)).sum(1).to(torch.bfloat16)


def _own(s):
    import token_dispatch_grouped_softmax_gb300 as moe

    c = s["case"]
    if c["op"] in ("route", "train"):
        how = dict(score=c["score"], n_groups=c["groups"], top_groups=c["top_groups"], group_score=c["group_score"],
                   renorm=c["renorm"], scale=c["scale"])
        ids, w = moe.route_select(s["logits"], c["k"], bias=s["bias"], **how)
        if c["op"] == "route":
            return dict(ids=ids, w=w)
        out = dict(ids=ids, w=w, d_logits=moe.route_select_bwd(s["dw"], s["logits"], ids, score=c["score"],
                                                              renorm=c["renorm"], scale=c["scale"]))
        if s["bias"] is not None:
            out["bias"] = moe.route_balance_bias(s["bias"], s["counts"], 0.001)
        return out
    if c["op"] == "gate_up":
        return moe.w4_gate_up_swiglu(s["x"], s["ids"], s["q"], s["scales"], s["zeros"])
    return moe.w4_down_combine(s["h"], s["ids"], s["w"], s["q"], s["scales"], s["zeros"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- what it is

def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] in ("route", "train"):
        es = 2 if c["dtype"] == "bf16" else 4
        b = T * E * es + T * k * 8 + (4 * E if c["bias"] else 0)
        f = 4 * T * E
        if c["op"] == "train":
            b += T * E * es + T * k * 4 + (8 * E if c["bias"] else 0)
            f += 4 * T * (E if c["score"] == "softmax" and not c["renorm"] else k)
        return dict(bytes=b, flops=f)
    K, N = _cols(c)
    rows = T - max(1, T // 8) if c["pad"] else T
    used = E * (1.0 - (1.0 - k / E) ** rows)     # distinct experts of `rows` tokens, each choosing k of E evenly
    b = used * (K * N / 2 + (K // c["group"]) * N * (3 if c["zeros"] else 2)) + T * k * 4
    b += T * K * 2 + T * k * (N // 2) * 2 if c["op"] == "gate_up" else T * k * (K * 2 + 4) + T * N * 2
    return dict(bytes=b, flops=2.0 * rows * k * K * N)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] in ("route", "train"):
        z = s["logits"].double()
        s64 = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
        value = s64 + (s["bias"].double() if c["bias"] else 0.0)
        if not c["bias"] and (c["groups"] == 1 or c["group_score"] == "max"):
            value = z
        per = E // c["groups"]
        table = value.view(T, c["groups"], per).sort(dim=2, descending=True).values
        strength = table[:, :, 0] if c["group_score"] == "max" or per == 1 else table[:, :, :2].sum(2)
        rank = torch.argsort(torch.argsort(strength, dim=1, descending=True, stable=True), 1)
        outside = (rank >= c["top_groups"]).unsqueeze(2).expand(T, c["groups"], per).reshape(T, E)
        ids = value.masked_fill(outside, -1e300).argsort(dim=1, descending=True, stable=True)[:, :k]
        onehot = torch.zeros_like(z).scatter_(1, ids, 1.0)
        chosen = s64 * onehot
        total = chosen.sum(1, keepdim=True) if c["renorm"] else torch.ones((T, 1), dtype=z.dtype, device=z.device)
        w = c["scale"] * (chosen / total)
        out = dict(ids=ids.to(torch.int32), w=w.gather(1, ids))
        if c["op"] == "route":
            return out
        # chain rule, one factor at a time: dw -> ds (chosen) -> dz
        up = torch.zeros_like(z).scatter_(1, ids, s["dw"].double())
        ds = c["scale"] * up / total
        if c["renorm"]:
            ds = ds - onehot * c["scale"] * (up * chosen).sum(1, keepdim=True) / total ** 2
        if c["score"] == "sigmoid":
            dz = ds * s64 * torch.sigmoid(-z)
        else:
            dz = s64 * (ds - (ds * s64).sum(1, keepdim=True))
        out["d_logits"] = dz
        if c["bias"]:
            load = s["counts"].double()
            out["bias"] = s["bias"].double() + 0.001 * torch.sign(load.mean() - load)
        return out
    K, N = _cols(c)
    G = c["group"]
    ids = s["ids"].view(-1)
    x = s["x"].double().repeat_interleave(k, 0) if c["op"] == "gate_up" else s["h"].double().view(T * k, K)
    y = torch.zeros((T * k, N), dtype=torch.float64, device=DEV)
    for e in sorted(set(ids.tolist()) - {-1}):
        word = s["q"][e * K // 8:(e + 1) * K // 8]
        w = torch.stack([(word >> (4 * i)).bitwise_and(15) for i in range(8)], 1).reshape(K, N).double()
        at = slice(e * K // G, (e + 1) * K // G)
        w -= 8.0 if s["zeros"] is None else s["zeros"][at].double().repeat_interleave(G, 0)
        w *= s["scales"][at].double().repeat_interleave(G, 0)
        here = (ids == e).nonzero().view(-1)
        y[here] = x[here] @ w
    if c["op"] == "gate_up":
        g, u = y[:, :c["I"]], y[:, c["I"]:]
        return (g * torch.sigmoid(g) * u).view(T, k, c["I"])
    return torch.einsum("tkn,tk->tn", y.view(T, k, N), s["w"].double())
