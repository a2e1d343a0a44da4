"""The MoE expert layer as a sequence of library calls, plus a torch autograd
Function around it.

Forward ("InternVL3.5 接入 pure FSDP2 后端开发实践", MindSpeed-MM issue 625,
§8.2-§8.3): route -> permute -> grouped gate_up GEMM + SwiGLU -> grouped down
GEMM -> unpermute-combine (+ the shared expert, "Awesome-ML-SYS-Tutorial"
MoE/EP guide: shared experts are always active).  All calls are enqueued on
the current stream with no host synchronisation: expert_offsets stay on the
device and the grouped GEMMs read them there.

Backward: combine_bwd (dY rows to permuted order) -> down_bwd -> route_bwd ->
gate_up_bwd -> gather_dx.
"""
from __future__ import annotations

import contextlib
import functools
from dataclasses import dataclass

import torch

from . import ops


def _range(name):
    """An NVTX range around one step of the layer, so that a profiler's
    timeline (Nsight Systems, Nsight Compute's NVTX filters) shows which
    library call enqueued each kernel; inside a CUDA graph capture the ranges
    mark the capture only."""
    nvtx = getattr(torch.cuda, "nvtx", None)
    return nvtx.range(name) if nvtx is not None else contextlib.nullcontext()


@dataclass(frozen=True)
class Routing:
    """How experts are chosen from the router's logits (ops.route_select):
    softmax or sigmoid scores, the best top_groups of n_groups groups of
    experts, weights renormalised over the chosen experts or not, and scaled.
    Without one (routing=None) the layer routes by ops.route."""
    score: str = "softmax"
    n_groups: int = 1
    top_groups: int = 1
    group_score: str = "top2"
    renorm: bool = True
    scale: float = 1.0

    @property
    def dense_gradient(self):
        """Whether the logits of experts that were not chosen have a gradient too."""
        return self.score == "softmax" and not self.renorm

    def select(self, logits, k, balance_bias=None):
        return ops.route_select(logits, k, balance_bias, self.score, self.n_groups, self.top_groups, self.group_score,
                                self.renorm, self.scale)


def _route(x, w_router, k, bias, w_split, routing, balance_bias):
    """ids, w and, with a Routing, the logits that they were chosen from."""
    if routing is None:
        if balance_bias is not None:
            raise ValueError("balance_bias needs a Routing")
        ids, w = ops.route(x, w_router, k, bias, w_split=w_split)
        return ids, w, None
    logits = ops.route_logits(x, w_router, bias, w_split)
    ids, w = routing.select(logits, k, balance_bias)
    return ids, w, logits


@dataclass
class ForwardState:
    """What the forward keeps for the backward."""
    x: torch.Tensor
    ids: torch.Tensor
    w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    row_map: torch.Tensor
    src_row: torch.Tensor
    h: torch.Tensor
    y_perm: torch.Tensor
    w_perm: torch.Tensor | None = None
    gu_pre: torch.Tensor | None = None     # fp32 [R, 2I]
    h_w: torch.Tensor | None = None        # bf16 w * h [R, I]
    x_perm: torch.Tensor | None = None     # bf16 [R, H] when the rows were materialised
    y_shared: torch.Tensor | None = None
    logits: torch.Tensor | None = None     # fp32 [T, E], with a Routing
    routing: Routing | None = None


def moe_forward(x, w_router, gate_up, down, k, bias=None, sh_gate_up=None, sh_down=None,
                save_for_backward=False, fused_gather=False, w_split=None, routing=None, balance_bias=None):
    """y [T, H] bf16 and the ForwardState.

    fused_gather: the grouped gate_up GEMM gathers the token rows itself (the
    permute fused into the operand load by TMA tile::gather4); False
    (default) materialises the permuted rows first (moe_permute_rows_scatter) and
    streams them with 128-row TMA tiles, which measures ~2.5x faster for the
    GEMM on GB300.
    w_split: W_r's bf16 split (ops.route_split_weight), prepared once while
    W_r does not change; the same results as without it.
    routing, balance_bias: a Routing, and the [E] fp32 bias that it adds to the
    scores for the choice alone (bias is added to the logits)."""
    T, H = x.shape
    E = w_router.shape[1]
    I = down.shape[0] // E
    if save_for_backward and routing is not None and routing.dense_gradient:
        raise ValueError("softmax without renorm has a gradient at every expert's logit, which the layer's backward "
                         "does not carry into dX (ops.route_select_bwd gives it)")
    with _range("moe.route"):
        ids, w, logits = _route(x, w_router, k, bias, w_split, routing, balance_bias)
    w_perm = None
    with _range("moe.permute"):
        if save_for_backward:
            counts, offsets, row_map, src_row, w_perm = ops.permute(ids, E, w)
        else:
            counts, offsets, row_map, src_row = ops.permute(ids, E)
    x_perm = None
    if fused_gather:
        with _range("moe.gate_up"):
            h, gu_pre, h_w = ops.grouped_gemm_gate_up_swiglu(x, src_row, offsets, gate_up, I, w_perm=w_perm,
                                                             save_for_backward=save_for_backward)
    else:
        with _range("moe.permute_rows"):
            x_perm = ops.permute_rows_scatter(x, row_map, k)
        with _range("moe.gate_up"):
            h, gu_pre, h_w = ops.grouped_gemm_gate_up_swiglu(x_perm, None, offsets, gate_up, I, w_perm=w_perm,
                                                             save_for_backward=save_for_backward)
    with _range("moe.down"):
        y_perm = ops.grouped_gemm_down(h, offsets, down, H)
    y_shared = None
    if sh_gate_up is not None:
        I_s = sh_down.shape[0]
        with _range("moe.shared_expert"):
            hs, _, _ = ops.grouped_gemm_gate_up_swiglu(x, None, None, sh_gate_up, I_s)
            y_shared = ops.grouped_gemm_down(hs, None, sh_down, H)
    with _range("moe.combine"):
        y = ops.unpermute_combine(y_perm, row_map, w, y_shared)
    st = ForwardState(x, ids, w, counts, offsets, row_map, src_row, h, y_perm, w_perm, gu_pre, h_w, x_perm,
                      y_shared, logits, routing)
    return y, st


def moe_backward(dy, st: ForwardState, w_router, gate_up, down, want_dw_router=False):
    """dict(dx, d_logits, d_gate_up, d_down, dw[, d_w_router]) for upstream gradient dy."""
    if st.gu_pre is None:
        raise ValueError("the forward ran without save_for_backward=True")
    T, H = st.x.shape
    E = w_router.shape[1]
    k = st.w.shape[1]
    with _range("moe.combine_bwd"):
        # dy_perm[row] = dY[src_row[row]], moved token by token (each dY row read
        # once; the same bits as ops.unpermute_combine_bwd, the gather)
        dy_perm = ops.permute_rows_scatter(dy, st.row_map, k)
    with _range("moe.down_bwd"):
        dgu, d_down, dw_part = ops.grouped_gemm_down_bwd(dy_perm, st.h_w, st.gu_pre, st.w_perm, st.offsets, down)
    with _range("moe.route_bwd"):
        if st.routing is None:
            d_logits, dw = ops.route_bwd(dw_part, st.row_map, st.w, st.ids, E)
        else:
            r = st.routing
            d_logits, dw = ops.route_select_bwd(dw_part, st.logits, st.ids, r.score, r.renorm, r.scale, st.row_map)
    with _range("moe.gate_up_bwd"):
        if st.x_perm is not None:
            dx_perm, d_gate_up = ops.grouped_gemm_gate_up_bwd(dgu, st.x_perm, None, st.offsets, gate_up)
        else:
            dx_perm, d_gate_up = ops.grouped_gemm_gate_up_bwd(dgu, st.x, st.src_row, st.offsets, gate_up)
    with _range("moe.gather_dx"):
        dx = ops.gather_dx(dx_perm, st.row_map, T, k, d_logits, st.ids, w_router)
    out = dict(dx=dx, d_logits=d_logits, d_gate_up=d_gate_up, d_down=d_down, dw=dw)
    if want_dw_router:
        with _range("moe.route_bwd_weight"):
            out["d_w_router"] = ops.route_bwd_weight(st.x, d_logits)
    return out


class _NoSecondDerivative(torch.autograd.Function):
    """Its arguments after the first as they are; differentiating them raises."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g.detach() for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the layer's and the norms' gradients cannot be differentiated again: their kernels record no graph")


def _first_order(backward):
    """For a Function's backward whose kernels record no graph: its gradients
    under create_graph=True raise when they are differentiated, where the terms
    through them would be missing.  (torch's once_differentiable does so only
    where the incoming gradient has a graph, which a sum's has not.)"""

    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = list(backward(ctx, *grads))
        given = [i for i, g in enumerate(out) if g is not None]
        if torch.is_grad_enabled() and given:
            for i, g in zip(given, _NoSecondDerivative.apply(torch.zeros((), requires_grad=True), *(out[i] for i in given))):
                out[i] = g
        return tuple(out)

    return run


class MoELayerFunction(torch.autograd.Function):
    """y = MoE(x); gradients for x, W_r, gate_up and down (fp32 W_r grad)."""

    @staticmethod
    def forward(ctx, x, w_router, gate_up, down, k, bias):
        y, st = moe_forward(x.contiguous(), w_router.contiguous(), gate_up.contiguous(),
                            down.contiguous(), k, bias, save_for_backward=True)
        ctx.st = st
        ctx.save_for_backward(w_router, gate_up, down)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        w_router, gate_up, down = ctx.saved_tensors
        g = moe_backward(dy.contiguous(), ctx.st, w_router, gate_up, down,
                         want_dw_router=ctx.needs_input_grad[1])
        return (g["dx"], g.get("d_w_router"), g["d_gate_up"], g["d_down"], None, None)


class RoutedMoELayerFunction(torch.autograd.Function):
    """MoELayerFunction with a Routing: y and the experts' loads (permute's
    counts, for ops.route_balance_bias).  The balance bias chooses only and has no gradient."""

    @staticmethod
    def forward(ctx, x, w_router, gate_up, down, k, bias, routing, balance_bias):
        y, st = moe_forward(x.contiguous(), w_router.contiguous(), gate_up.contiguous(), down.contiguous(), k, bias,
                            save_for_backward=True, routing=routing, balance_bias=balance_bias)
        ctx.st = st
        ctx.save_for_backward(w_router, gate_up, down)
        ctx.mark_non_differentiable(st.counts)
        return y, st.counts

    @staticmethod
    @_first_order
    def backward(ctx, dy, _):
        w_router, gate_up, down = ctx.saved_tensors
        g = moe_backward(dy.contiguous(), ctx.st, w_router, gate_up, down, want_dw_router=ctx.needs_input_grad[1])
        return (g["dx"], g.get("d_w_router"), g["d_gate_up"], g["d_down"], None, None, None, None)


class MoELayer(torch.nn.Module):
    """Routed SwiGLU experts over the fused layout gate_up [E*H, 2I], down [E*I, H].

    routing: a Routing; the layer then holds a balance bias (a buffer, zeros at
    first) that update_balance_bias moves by the loads of the last forward.
    With a bias, of zeros too, the rounded scores plus the bias choose;
    balance=False holds none, and where the scores order the experts as the
    logits do, the logits choose, as in moe_forward without a bias.  A
    Routing with a dense gradient (softmax without renorm) runs where no
    gradient is asked for and is refused where one is."""

    def __init__(self, hidden: int, n_experts: int, top_k: int, inter: int, device="cuda", routing=None, balance=True):
        super().__init__()
        if routing is None and not balance:
            raise ValueError("balance=False needs a Routing")
        self.k = top_k
        self.routing = routing
        if routing is not None:
            bias = torch.zeros(n_experts, dtype=torch.float32, device=device) if balance else None
            self.register_buffer("balance_bias", bias)
            self.last_counts = None
        self.w_router = torch.nn.Parameter(torch.empty(hidden, n_experts, dtype=torch.float32, device=device))
        self.gate_up = torch.nn.Parameter(torch.empty(n_experts * hidden, 2 * inter, dtype=torch.bfloat16,
                                                      device=device))
        self.down = torch.nn.Parameter(torch.empty(n_experts * inter, hidden, dtype=torch.bfloat16,
                                                   device=device))

    def forward(self, x, bias=None):
        if self.routing is not None:
            weights = (self.w_router, self.gate_up, self.down)
            if torch.is_grad_enabled() and any(t.requires_grad for t in (x,) + weights):
                y, self.last_counts = RoutedMoELayerFunction.apply(x, *weights, self.k, bias, self.routing,
                                                                   self.balance_bias)
            else:   # nothing is kept for a backward, and a Routing with a dense gradient runs too
                y, st = moe_forward(x.contiguous(), *(t.contiguous() for t in weights), self.k, bias,
                                    routing=self.routing, balance_bias=self.balance_bias)
                self.last_counts = st.counts
            return y
        return MoELayerFunction.apply(x, self.w_router, self.gate_up, self.down, self.k, bias)

    @torch.no_grad()
    def decode(self, x, bias=None):
        """y of a few tokens (at most 128) in two launches (moe_forward_few);
        nothing is kept for a backward or for the balance bias."""
        return moe_forward_few(x.contiguous(), self.w_router, self.gate_up, self.down, self.k, bias, routing=self.routing,
                               balance_bias=None if self.routing is None else self.balance_bias)[0]

    def update_balance_bias(self, rate):
        """balance_bias += rate * sign(mean load - load) by the last forward's loads."""
        if self.routing is None or self.balance_bias is None or self.last_counts is None:
            raise ValueError("update_balance_bias needs a layer with a Routing and a balance bias, after a forward")
        ops.route_balance_bias(self.balance_bias, self.last_counts, rate, out=self.balance_bias)


class BlockNormFunction(torch.autograd.Function):
    """ops.block_norm as (r, h) with its gradients; an operand that is None has none."""

    @staticmethod
    def forward(ctx, x, weight, branch, post_weight, gate, residual_scale, branch_scale, eps):
        t = [None if v is None else v.contiguous() for v in (x, weight, branch, post_weight, gate)]
        r, h, stats = ops.block_norm(t[0], t[1], t[2], t[3], t[4], residual_scale, branch_scale, eps, save_for_backward=True)
        ctx.save_for_backward(*t, stats)
        ctx.scales = residual_scale, branch_scale
        ctx.set_materialize_grads(False)
        return r, h

    @staticmethod
    @_first_order
    def backward(ctx, dr, dh):
        x, weight, branch, post_weight, gate, stats = ctx.saved_tensors
        if weight is None:
            dh = None
        elif dh is None:
            dh = torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
        else:
            dh = dh.contiguous()
        dr = dr.contiguous() if dr is not None and branch is not None else None
        g = ops.block_norm_bwd(dh, dr, x, stats, weight, branch, post_weight, gate, *ctx.scales)
        return g["dx"], g["d_weight"], g["d_branch"], g["d_post_weight"], g["d_gate"], None, None, None


def block_norm_autograd(x, weight=None, branch=None, post_weight=None, gate=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6):
    """(r, h) of ops.block_norm, with gradients for the operands that ask for
    them: the norms outside a MoEBlock, such as the one after the last block,
    ``block_norm_autograd(x, weight)[1]``."""
    given = (x, weight, branch, post_weight, gate)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in given):
        return BlockNormFunction.apply(*given, residual_scale, branch_scale, eps)
    t = [None if v is None else v.contiguous() for v in given]
    return ops.block_norm(*t, residual_scale, branch_scale, eps)[:2]


block_norm = block_norm_autograd   # in this module; the package's block_norm is ops.block_norm


class MoEBlock(torch.nn.Module):
    """A model's block around a MoELayer: the residual stream normed, the
    layer, and its output added to the stream, by default as it is:

        r = residual_scale x + branch_scale gate norm(layer(norm(x)))

    post_norm norms the layer's output, learned_scale multiplies it by a
    learned [H] vector, and forward takes a gate of its own (block_norm's).
    The stream is fp32 or bf16; the layer runs in bf16.  A run of blocks fuses
    each block's end with the next one's norm: ``r, h = block(x, h,
    next_norm=following.norm)``."""

    def __init__(self, layer, eps=1e-6, post_norm=False, learned_scale=None, residual_scale=1.0, branch_scale=1.0):
        super().__init__()
        H, device = layer.w_router.shape[0], layer.w_router.device
        self.layer, self.eps = layer, eps
        self.residual_scale, self.branch_scale = residual_scale, branch_scale
        vector = lambda v: torch.nn.Parameter(torch.full((H,), float(v), dtype=torch.float32, device=device))
        self.norm = vector(1.0)
        self.post_norm = vector(1.0) if post_norm else None
        self.scale = vector(learned_scale) if learned_scale is not None else None

    def _around(self, run, x, h, next_norm, gate):
        if self.scale is not None:
            if gate is not None:
                raise ValueError("a block with a learned scale takes no gate")
            gate = self.scale.unsqueeze(0)
        if h is None:
            h = block_norm_autograd(x, self.norm, eps=self.eps)[1]
        return block_norm_autograd(x, next_norm, run(h), self.post_norm, gate, self.residual_scale, self.branch_scale, self.eps)

    def forward(self, x, h=None, next_norm=None, gate=None, bias=None):
        """(r, h of the next block or None): x [T, H] the stream, h the stream
        normed already (by the block before), next_norm the next block's norm
        weight, bias the layer's."""
        return self._around(lambda t: self.layer(t, bias), x, h, next_norm, gate)

    @torch.no_grad()
    def decode(self, x, h=None, next_norm=None, gate=None, bias=None):
        """forward of a few tokens through MoELayer.decode."""
        return self._around(lambda t: self.layer.decode(t, bias), x, h, next_norm, gate)


@torch.no_grad()
def clip_grad_norm(parameters, max_norm, eps=1e-6):
    """Scales the parameters' gradients in place so that their 2-norm is at
    most max_norm, and returns the norm they had (ops.clip_grads); parameters
    without a gradient are left out, one that is given twice counts once; none
    with a gradient is a ValueError.  A gradient may have any dense layout, as
    that of a transposed parameter."""
    grads = list({id(p): p.grad for p in parameters if p.grad is not None}.values())
    return ops.clip_grads(grads, max_norm, eps=eps)


@dataclass
class BF16Experts:
    """The experts' weights in bf16: gate_up [E*H, 2I], down [E*I, H] and the number of experts."""
    gate_up: torch.Tensor
    down: torch.Tensor
    n_experts: int


@dataclass
class W4Experts:
    """The experts' weights in 4 bits: gate_up and down as (qweight, scales,
    zeros or None) of ops.w4_quantize, with the number of experts."""
    gate_up: tuple
    down: tuple
    n_experts: int

    @classmethod
    def quantize(cls, gate_up, down, n_experts, group=128, zeros=False):
        """From gate_up [E*H, 2I] and down [E*I, H] in bf16."""
        return cls(ops.w4_quantize(gate_up, group, zeros), ops.w4_quantize(down, group, zeros), n_experts)

    def dequantize(self):
        """gate_up and down in bf16."""
        return ops.w4_dequantize(*self.gate_up), ops.w4_dequantize(*self.down)


# From this many rows an expert on, the 4-bit kernels' chunks of 8 rows (each
# of which decodes the weights again) cost more than one decoding to bf16 and
# the bf16 grouped GEMMs: measured equal at 48 rows (H 2048, E 128, I 768), 51
# (H 4096, E 8, I 2048) and 32 (H 7168, E 256, I 2048).  A value for
# moe_forward_w4's bf16_rows.
W4_MAX_ROWS_PER_EXPERT = 48


def _decoded_experts(x, gate_up, down, offsets=None):
    """x's rows (permuted, or with offsets None all of one expert's) through
    4-bit weights that are decoded to bf16, one of the two at a time."""
    weight = ops.w4_dequantize(*gate_up)
    h, _, _ = ops.grouped_gemm_gate_up_swiglu(x, None, offsets, weight, weight.shape[1] // 2)
    del weight
    return ops.grouped_gemm_down(h, offsets, ops.w4_dequantize(*down), x.shape[1])


def moe_forward_w4(x, w_router, experts, k, bias=None, shared=None, w_split=None, routing=None, balance_bias=None,
                   bf16_rows=None):
    """y [T, H] bf16 through 4-bit experts (W4Experts), and the slots' ids and w.

    route -> gate_up + SwiGLU -> down + combine, rows in slot order with no
    permutation; a token's result does not depend on the batch.  shared: a
    W4Experts of one expert, always active.

    bf16_rows: where there are more rows per expert (T*k / E) than this, decode
    the weights to bf16 for the call and run moe_forward's grouped GEMMs on
    them, and the shared expert's from twice as many tokens on.  That is faster from
    W4_MAX_ROWS_PER_EXPERT on and less exact: the weights and each slot's
    product are rounded to bf16.  It takes the larger of gate_up's E*H*2I and
    down's E*I*H bf16 weights of memory for the call.  None: never."""
    T, H = x.shape
    E = experts.n_experts
    if w_router.shape[1] != E:
        raise ValueError("w_router must be [H, E] for the experts' E")
    with _range("moe.route"):
        ids, w, _ = _route(x, w_router, k, bias, w_split, routing, balance_bias)
    y_shared = None
    if shared is not None:
        with _range("moe.shared_expert"):
            if bf16_rows is not None and T > 2 * bf16_rows:   # one expert's launches: equal at 95 (I 2048) to 250 rows (H 2048, I 768)
                y_shared = _decoded_experts(x, shared.gate_up, shared.down)
            else:
                y_shared = ops.w4_down_combine(ops.w4_gate_up_swiglu(x, None, *shared.gate_up), None, None, *shared.down)
    if bf16_rows is not None and T * k > bf16_rows * E:
        with _range("moe.permute"):
            _, offsets, row_map, _ = ops.permute(ids, E)
        with _range("moe.permute_rows"):
            x_perm = ops.permute_rows_scatter(x, row_map, k)
        with _range("moe.experts"):
            y_perm = _decoded_experts(x_perm, experts.gate_up, experts.down, offsets)
        with _range("moe.combine"):
            return ops.unpermute_combine(y_perm, row_map, w, y_shared), ids, w
    with _range("moe.gate_up"):
        h = ops.w4_gate_up_swiglu(x, ids, *experts.gate_up)
    with _range("moe.down"):
        return ops.w4_down_combine(h, ids, w, *experts.down, y_shared=y_shared), ids, w


def moe_forward_few(x, w_router, gate_up, down, k, bias=None, sh_gate_up=None, sh_down=None, routing=None,
                    balance_bias=None):
    """y [T, H] bf16 of a few tokens (T at most 128) through bf16 experts, and the slots' ids and w: the layer of a decode step, as
    moe_forward_w4 for weights that are not quantised.  Rows stay in slot
    order, the experts' products in fp32 until the tokens' sums; a token's
    result does not depend on the batch."""
    if routing is None:
        if balance_bias is not None:
            raise ValueError("balance_bias needs a Routing")
        routing = Routing()
    return ops.layer_few(x, w_router, gate_up, down, k, bias, balance_bias, sh_gate_up, sh_down, routing.score,
                         routing.n_groups, routing.top_groups, routing.group_score, routing.renorm, routing.scale)


class DecodeGraph:
    """A decode step captured once as a CUDA graph for a fixed token count:
    moe_forward_w4 for W4Experts, moe_forward_few for BF16Experts (at most 128
    tokens).  Write a step's tokens into ``x`` (or pass them to ``__call__``);
    a replay is one launch and writes ``y``, ``ids`` and ``w``, which the next
    replay overwrites.  Routing stays on the device, so one capture serves any
    routing.  As ForwardGraph, with 4-bit experts it makes W_r's bf16 split once
    (``refresh_router_split()`` after changing W_r); with bf16 ones W_r is read
    as it is."""

    def __init__(self, T, w_router, experts, k, bias=None, shared=None, routing=None, balance_bias=None, bf16_rows=None):
        H, E = w_router.shape
        self.args = (w_router, experts, k, bias, shared)
        self.routing, self.balance_bias, self.bf16_rows = routing, balance_bias, bf16_rows
        self.few = isinstance(experts, BF16Experts)
        if self.few and (bf16_rows is not None or not (shared is None or isinstance(shared, BF16Experts))):
            raise ValueError("bf16 experts take a shared expert in bf16 and no bf16_rows")
        if self.few and experts.n_experts != E:
            raise ValueError("w_router must be [H, E] for the experts' E")
        self.w_split = ops.route_split_weight(w_router) if not self.few and ops.route_supports_split(H, E) else None
        self.x = torch.zeros((T, H), dtype=torch.bfloat16, device=w_router.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):          # one-time library set-up happens outside the capture
            for _ in range(2):
                self._forward()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y, self.ids, self.w = self._forward()

    def _forward(self):
        if self.few:
            w_router, experts, k, bias, shared = self.args
            sh = (shared.gate_up, shared.down) if shared is not None else (None, None)
            return moe_forward_few(self.x, w_router, experts.gate_up, experts.down, k, bias, *sh, self.routing, self.balance_bias)
        return moe_forward_w4(self.x, *self.args, w_split=self.w_split, routing=self.routing,
                              balance_bias=self.balance_bias, bf16_rows=self.bf16_rows)

    def refresh_router_split(self):
        """Re-derives W_r's split (in place, where the graph reads it) after W_r changed."""
        if self.w_split is not None:
            ops.route_split_weight(self.args[0], out=self.w_split)

    def replay(self):
        """Runs the layer on the current contents of ``x``; returns ``y``."""
        self.graph.replay()
        return self.y

    def __call__(self, x):
        self.x.copy_(x)
        return self.replay()


class ForwardGraph:
    """The layer forward captured once as a CUDA graph, for a fixed token
    count and fixed weights (inference).

    Write a batch's tokens into ``x`` (or pass them to ``__call__``); a replay
    runs route, permute, both grouped GEMMs and the combine as one graph
    launch, with no per-kernel launch gaps, and writes ``y``, which the next
    replay overwrites.  Every step of the path stays on the device (expert
    offsets included), so one capture serves any routing.  The graph keeps
    its intermediates in its own memory pool.

    The weights are fixed for the graph's life: W_r's bf16 split (the tensor
    cores' router operand) is made once here, outside the graph.  After
    changing W_r in place, call ``refresh_router_split()``.
    """

    def __init__(self, T, w_router, gate_up, down, k, bias=None, sh_gate_up=None, sh_down=None,
                 fused_gather=False):
        H, E = w_router.shape
        self.args = (w_router, gate_up, down, k, bias, sh_gate_up, sh_down)
        self.fused_gather = fused_gather
        self.w_split = ops.route_split_weight(w_router) if ops.route_supports_split(H, E) else None
        self.x = torch.zeros((T, H), dtype=torch.bfloat16, device=w_router.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):          # one-time library set-up happens outside the capture
            for _ in range(2):
                self._forward()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self._forward()

    def _forward(self):
        w_router, gate_up, down, k, bias, sh_gu, sh_dn = self.args
        y, _ = moe_forward(self.x, w_router, gate_up, down, k, bias, sh_gu, sh_dn,
                           fused_gather=self.fused_gather, w_split=self.w_split)
        return y

    def refresh_router_split(self):
        """Re-derives W_r's split (in place, where the graph reads it) after W_r changed."""
        if self.w_split is not None:
            ops.route_split_weight(self.args[0], out=self.w_split)

    def replay(self):
        """Runs the layer on the current contents of ``x``; returns ``y``."""
        self.graph.replay()
        return self.y

    def __call__(self, x):
        self.x.copy_(x)
        return self.replay()


class PipelinedForward:
    """The forward over a stream of host batches, with copies overlapped.

    Batch i's layer runs on the compute stream while batch i+1's tokens are
    copied host -> device and batch i-1's output device -> host on a copy
    stream (events between the streams).  The layer runs as one of two
    ForwardGraph replays, one per input buffer.  Host tensors must be pinned
    for the copies to be asynchronous; every batch has the token count the
    graphs were captured for.
    """

    def __init__(self, T, w_router, gate_up, down, k, bias=None, sh_gate_up=None, sh_down=None,
                 fused_gather=False):
        self.graphs = [ForwardGraph(T, w_router, gate_up, down, k, bias, sh_gate_up, sh_down,
                                    fused_gather) for _ in range(2)]
        self.copy_stream = torch.cuda.Stream()
        self.ev_loaded = [torch.cuda.Event(), torch.cuda.Event()]
        self.ev_done = [torch.cuda.Event(), torch.cuda.Event()]
        self.ev_stored = [torch.cuda.Event(), torch.cuda.Event()]

    def run(self, x_host_batches, y_host_batches):
        """y_host_batches[i] <- layer(x_host_batches[i]); returns when all are stored."""
        compute = torch.cuda.current_stream()
        n = len(x_host_batches)
        for b in range(2):
            self.ev_done[b].record(compute)     # both buffers free at the start
            self.ev_stored[b].record(compute)

        def load(i):
            b = i % 2
            with torch.cuda.stream(self.copy_stream):
                self.copy_stream.wait_event(self.ev_done[b])     # the layer no longer reads it
                self.graphs[b].x.copy_(x_host_batches[i], non_blocking=True)
                self.ev_loaded[b].record(self.copy_stream)

        if n:
            load(0)
        for i in range(n):
            b = i % 2
            if i + 1 < n:
                load(i + 1)
            compute.wait_event(self.ev_loaded[b])
            compute.wait_event(self.ev_stored[b])                # batch i-2's output was copied out
            y = self.graphs[b].replay()
            self.ev_done[b].record(compute)
            with torch.cuda.stream(self.copy_stream):
                self.copy_stream.wait_event(self.ev_done[b])
                y_host_batches[i].copy_(y, non_blocking=True)
                self.ev_stored[b].record(self.copy_stream)
        self.copy_stream.synchronize()
        compute.synchronize()


class OverlappedForward:
    """The forward over a stream of host batches as a two-stage pipeline, so
    that the token-side steps of one batch overlap the expert GEMMs of the
    previous one (the single-GPU part of the Domino-style overlap: ByteDance
    "FSDPTurbo" domino dispatcher; "InternVL3.5 pure FSDP2 训练性能优化实践").

    Stage F (route -> permute -> row gather) and stage G (grouped gate_up
    GEMM -> grouped down GEMM -> combine, plus the shared expert) are each
    captured as a CUDA graph per buffer set, two sets, and run on their own
    streams: F of batch i+1 runs while G of batch i runs.  Tokens are not
    split within a batch, so every expert's weights are still read once per
    batch.  A copy stream uploads each batch and downloads its output.
    Outputs equal moe_forward's bit for bit.  Host tensors must be pinned;
    every batch has the token count given here.  As ForwardGraph, it makes
    W_r's bf16 split once at construction (``refresh_router_split()`` after
    changing W_r).
    """

    def __init__(self, T, w_router, gate_up, down, k, bias=None, sh_gate_up=None, sh_down=None,
                 fused_gather=False):
        H, E = w_router.shape
        I = down.shape[0] // E
        self.w_router = w_router
        self.w_split = ops.route_split_weight(w_router) if ops.route_supports_split(H, E) else None
        w_split = self.w_split
        self.stream_f = torch.cuda.Stream()
        self.stream_g = torch.cuda.Stream()
        self.copy_stream = torch.cuda.Stream()
        # stage G reads x itself for the shared expert and the fused row gather
        self.g_reads_x = sh_gate_up is not None or fused_gather
        self.sets = []
        for _ in range(2):
            st = {"x": torch.zeros((T, H), dtype=torch.bfloat16, device=w_router.device)}

            def front(st=st):
                ids, w = ops.route(st["x"], w_router, k, bias, w_split=w_split)
                counts, offsets, row_map, src_row = ops.permute(ids, E)
                x_perm = None if fused_gather else ops.permute_rows_scatter(st["x"], row_map, k)
                st.update(w=w, offsets=offsets, row_map=row_map, src_row=src_row, x_perm=x_perm)

            def back(st=st):
                if fused_gather:
                    h, _, _ = ops.grouped_gemm_gate_up_swiglu(st["x"], st["src_row"], st["offsets"], gate_up, I)
                else:
                    h, _, _ = ops.grouped_gemm_gate_up_swiglu(st["x_perm"], None, st["offsets"], gate_up, I)
                y_perm = ops.grouped_gemm_down(h, st["offsets"], down, H)
                y_sh = None
                if sh_gate_up is not None:
                    I_s = sh_down.shape[0]
                    hs, _, _ = ops.grouped_gemm_gate_up_swiglu(st["x"], None, None, sh_gate_up, I_s)
                    y_sh = ops.grouped_gemm_down(hs, None, sh_down, H)
                st["y"] = ops.unpermute_combine(y_perm, st["row_map"], st["w"], y_sh)

            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):      # one-time library set-up outside the captures
                for _ in range(2):
                    front()
                    back()
            torch.cuda.current_stream().wait_stream(side)
            st["gf"], st["gg"] = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            # The two stages run side by side: captured without programmatic
            # dependent launch, whose early-resident kernels would take the
            # SMs that the other stage fills at each GEMM's tail.
            pdl = ops.pdl_enabled()
            ops.set_pdl(False)
            try:
                with torch.cuda.graph(st["gf"]):
                    front()
                with torch.cuda.graph(st["gg"]):
                    back()
            finally:
                ops.set_pdl(pdl)
            st.update(ev_loaded=torch.cuda.Event(), ev_f=torch.cuda.Event(), ev_g=torch.cuda.Event(),
                      ev_stored=torch.cuda.Event())
            self.sets.append(st)

    def refresh_router_split(self):
        """Re-derives W_r's split (in place, where the graphs read it) after W_r changed."""
        if self.w_split is not None:
            ops.route_split_weight(self.w_router, out=self.w_split)

    def run(self, x_host_batches, y_host_batches):
        """y_host_batches[i] <- layer(x_host_batches[i]); returns when all are stored."""
        cur = torch.cuda.current_stream()
        for st in self.sets:                    # every buffer free at the start
            for ev in ("ev_f", "ev_g", "ev_stored"):
                st[ev].record(cur)
        for s in (self.stream_f, self.stream_g, self.copy_stream):
            s.wait_stream(cur)
        n = len(x_host_batches)

        def load(i):
            st = self.sets[i % 2]
            with torch.cuda.stream(self.copy_stream):
                self.copy_stream.wait_event(st["ev_f"])          # F of batch i-2 has read x
                if self.g_reads_x:
                    self.copy_stream.wait_event(st["ev_g"])      # and so has G of batch i-2
                st["x"].copy_(x_host_batches[i], non_blocking=True)
                st["ev_loaded"].record(self.copy_stream)

        if n:
            load(0)
        for i in range(n):
            st = self.sets[i % 2]
            if i + 1 < n:
                load(i + 1)
            with torch.cuda.stream(self.stream_f):
                self.stream_f.wait_event(st["ev_loaded"])
                self.stream_f.wait_event(st["ev_g"])             # G of batch i-2 no longer reads this set
                st["gf"].replay()
                st["ev_f"].record(self.stream_f)
            with torch.cuda.stream(self.stream_g):
                self.stream_g.wait_event(st["ev_f"])
                self.stream_g.wait_event(st["ev_stored"])        # batch i-2's output was copied out
                st["gg"].replay()
                st["ev_g"].record(self.stream_g)
            with torch.cuda.stream(self.copy_stream):
                self.copy_stream.wait_event(st["ev_g"])
                y_host_batches[i].copy_(st["y"], non_blocking=True)
                st["ev_stored"].record(self.copy_stream)
        self.copy_stream.synchronize()
        cur.wait_stream(self.stream_f)
        cur.wait_stream(self.stream_g)
        cur.synchronize()
