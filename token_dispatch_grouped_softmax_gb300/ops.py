"""Per-step entry points of the MoE layer on torch CUDA tensors.

Argument marshalling only: each function checks dtypes and shapes, allocates
its outputs with torch (device memory), and calls the matching C entry point
of libmoe_gb300.so on the current torch stream.  Every step runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import binding, call

_BF16 = torch.bfloat16


# The current device and its current stream's handle without torch's wrapper
# objects (3 us a call on GB300's host) where this torch has the raw accessors.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the path runs only on the GPU)" % name)
    if t.get_device() != _current_device():
        # the kernels run on the current device and would be handed another GPU's memory
        raise ValueError("%s is on %s but the current device is cuda:%d" % (name, t.device, _current_device()))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims" % (name, ndim))
    return t


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def sync_status():
    """Synchronise the current stream and raise if a kernel reported a device-side error."""
    detail = ctypes.c_uint32(0)
    call("moe_sync_status", _stream(), ctypes.byref(detail))
    return detail.value


def set_wait_limit_ns(ns: int):
    call("moe_set_wait_limit_ns", int(ns))


GEMM_PAIRS_NONE, GEMM_PAIRS_ALL, GEMM_PAIRS_GATE_UP, GEMM_PAIRS_GATE_UP_WGRAD = 0, 1, 2, 3


def set_gemm_pairs(mode):
    """Where the grouped GEMMs run: False / GEMM_PAIRS_NONE on single CTAs,
    True / GEMM_PAIRS_ALL every forward and dgrad GEMM on CTA pairs (2-SM
    MMAs), GEMM_PAIRS_GATE_UP the forward gate_up GEMM on pairs,
    GEMM_PAIRS_GATE_UP_WGRAD that and the two weight-gradient GEMMs.  The
    results are bit-identical."""
    call("moe_set_gemm_pairs", int(mode))


_pdl_on = [True]


def set_pdl(on: bool):
    """Programmatic dependent launch of every kernel (default on): a kernel's
    set-up overlaps the tail of the one before it on the stream.  Off for
    graphs whose kernels run beside another stream's (OverlappedForward)."""
    call("moe_set_pdl", 1 if on else 0)
    _pdl_on[0] = bool(on)


def pdl_enabled() -> bool:
    """The setting last made through set_pdl (the library starts with it on)."""
    return _pdl_on[0]


# ----------------------------------------------------------------- forward

def route(x, w_router, k, bias=None, return_logits=False, w_split=None):
    """ids [T,k] int32, w [T,k] fp32 (and logits [T,E] fp32).

    w_split: W_r's bf16 split from route_split_weight(w_router), made once
    while W_r does not change (moe_route_presplit); the results are the same
    bit for bit."""
    _need(x, "x", _BF16, 2)
    _need(w_router, "w_router", torch.float32, 2)
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    T, H = x.shape
    E = w_router.shape[1]
    dev = x.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if return_logits else None
    nbytes = ctypes.c_size_t(0)
    if w_split is not None:
        _need(w_split, "w_split", _BF16, 2)
        if tuple(w_split.shape) != (3 * H, E):
            raise ValueError("w_split must be [3H, E] (route_split_weight)")
        call("moe_route_presplit_workspace_size", T, H, E, ctypes.byref(nbytes))
        ws = _ws(nbytes.value, dev) if nbytes.value else None
        call("moe_route_presplit", _p(x), _p(w_split), _p(bias), T, H, E, k, _p(ids), _p(w), _p(logits), _p(ws),
             ws.numel() if ws is not None else 0, _stream())
        return (ids, w, logits) if return_logits else (ids, w)
    call("moe_route_workspace_size", T, H, E, ctypes.byref(nbytes))
    ws = _ws(nbytes.value, dev)
    call("moe_route", _p(x), _p(w_router), _p(bias), T, H, E, k, _p(ids), _p(w), _p(logits), _p(ws),
         ws.numel(), _stream())
    return (ids, w, logits) if return_logits else (ids, w)


def route_supports_split(H, E):
    """Whether the router runs on the tensor cores at this shape (E % 8 == 0,
    H % 64 == 0, E <= 1024), the shapes route_split_weight serves."""
    return E % 8 == 0 and H % 64 == 0 and E <= 1024


def route_split_weight(w_router, out=None):
    """W_r's exact three-term bf16 split [3H, E] (W0 rows, then W1, then W2),
    for route(..., w_split=...) while W_r does not change.  out: an existing
    [3H, E] bf16 tensor to refresh in place (e.g. one a captured graph reads)."""
    _need(w_router, "w_router", torch.float32, 2)
    H, E = w_router.shape
    w_split = torch.empty((3 * H, E), dtype=_BF16, device=w_router.device) if out is None else out
    _need(w_split, "w_split", _BF16, 2)
    if tuple(w_split.shape) != (3 * H, E):
        raise ValueError("w_split must be [3H, E]")
    call("moe_route_split_weight", _p(w_router), H, E, _p(w_split), _stream())
    return w_split


# ----------------------------------------------------------- expert choice

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


def _choice(table, value, name):
    if value not in table:
        raise ValueError("%s must be one of %s" % (name, ", ".join(sorted(table))))
    return table[value]


# The functions up to w4_down_combine, and those of a decode step's bf16
# experts, a block's norms and the gradients' norm, check their tensors, allocate and call
# in the extension _binding (csrc/binding.cpp): a decode step's kernels run for
# a few microseconds, less than the same done in Python.

def route_logits(x, w_router, bias=None, w_split=None):
    """The router's logits [T, E] fp32 alone (moe_route), for route_select."""
    return route(x, w_router, 1, bias, return_logits=True, w_split=w_split)[2]


def route_select(logits, k, bias=None, score="softmax", n_groups=1, top_groups=1, group_score="top2", renorm=True,
                 scale=1.0):
    """ids [T, k] int32 and w [T, k] fp32 chosen from logits [T, E] (fp32 or bf16).

    score "softmax" or "sigmoid"; bias [E] fp32 is added to the scores for the
    choice alone; the top_groups best of n_groups groups of E / n_groups
    consecutive experts take part, a group's value being its best expert's
    ("max") or the sum of its two best ("top2"); renorm divides the chosen
    scores by their sum; scale multiplies them.  A logit of -inf masks its
    expert.  Equal values go to the lower index (moe_route_select)."""
    return binding().route_select(logits, k, bias, _choice(_SCORES, score, "score"), n_groups, top_groups,
                                  _choice(_GROUP_SCORES, group_score, "group_score"), bool(renorm), scale)


def route_select_bwd(dw, logits, ids, score="softmax", renorm=True, scale=1.0, row_map=None):
    """d_logits [T, E] of logits' type: the gradient of route_select's w for
    upstream dw [T, k] fp32, the choice held fixed.

    With row_map [T*k], dw is dw_part [T*k, nparts] from
    grouped_gemm_down_bwd (permuted rows, summed here), and (d_logits, dw
    [T, k]) is returned.  Softmax without renorm has a dense gradient."""
    return binding().route_select_bwd(dw, logits, ids, _choice(_SCORES, score, "score"), bool(renorm), scale, row_map)


def route_balance_bias(bias, counts, rate, out=None):
    """bias + rate * sign(mean load - load) [E] fp32, the loads being permute's
    counts [E] int32; out: an existing [E] fp32 tensor (bias itself to update in place)."""
    return binding().route_balance_bias(bias, counts, rate, out)


# ----------------------------------------------------------- 4-bit experts

def w4_gate_up_swiglu(x, ids, qweight, scales, zeros=None):
    """h [T, k, I] bf16 with h[t, j] = silu(x_t . Wg) * (x_t . Wu) of the 4-bit
    expert ids[t, j] (an id of -1: an empty slot, h = 0); rows in slot order.

    qweight [E*H/8, 2I] int32 (eight 4-bit codes of consecutive rows per
    word, lowest nibble first), scales [E*H/group, 2I] bf16, zeros of the same
    shape uint8 or None for 8 (w4_quantize makes them).  ids None: one dense
    expert."""
    return binding().w4_gate_up_swiglu(x, ids, qweight, scales, zeros)


def w4_down_combine(h, ids, w, qweight, scales, zeros=None, y_shared=None, out=None):
    """y [T, H] bf16 with y_t = sum_j w[t, j] (h[t, j] . Wd) (+ y_shared_t), e =
    ids[t, j] (-1 adds nothing); h [T, k, I] bf16 in slot order, w [T, k] fp32
    (None: 1), qweight [E*I/8, H] and scales [E*I/group, H] as in
    w4_gate_up_swiglu.  ids None: one dense expert."""
    return binding().w4_down_combine(h, ids, w, qweight, scales, zeros, y_shared, out)


def w4_quantize(weight, group=128, zeros=False):
    """(qweight [rows/8, N] int32, scales [rows/group, N] bf16, zeros uint8 or
    None) of bf16 weights [rows, N] (gate_up [E*H, 2I] or down [E*I, H]),
    group rows of a column sharing a scale (and a zero point with zeros=True)."""
    _need(weight, "weight", _BF16, 2)
    rows, N = weight.shape
    if group not in (32, 64, 128) or rows % group:
        raise ValueError("group must be 32, 64 or 128 and divide the rows")
    dev = weight.device
    q = torch.empty((rows // 8, N), dtype=torch.int32, device=dev)
    scales = torch.empty((rows // group, N), dtype=_BF16, device=dev)
    z = torch.empty((rows // group, N), dtype=torch.uint8, device=dev) if zeros else None
    call("moe_w4_quantize", _p(weight), rows, N, group, _p(q), _p(scales), _p(z), _stream())
    return q, scales, z


def w4_dequantize(qweight, scales, zeros=None):
    """bf16 weights [rows, N] of w4_quantize's layout: scale * (code - zero), one rounding."""
    _need(qweight, "qweight", torch.int32, 2)
    _need(scales, "scales", _BF16, 2)
    rows, N = qweight.shape[0] * 8, qweight.shape[1]
    if scales.shape[1] != N or scales.shape[0] == 0 or rows % scales.shape[0]:
        raise ValueError("scales must be [rows/group, N]")
    group = rows // scales.shape[0]
    if zeros is not None:
        _need(zeros, "zeros", torch.uint8, 2)
        if zeros.shape != scales.shape:
            raise ValueError("zeros must be [rows/group, N]")
    w = torch.empty((rows, N), dtype=_BF16, device=qweight.device)
    call("moe_w4_dequantize", _p(qweight), _p(scales), _p(zeros), rows, N, group, _p(w), _stream())
    return w


# ------------------------------------------- the layer for a few tokens

def experts_few(x, ids, w, gate_up, down, sh_gate_up=None, sh_down=None, out=None):
    """y [T, H] bf16 with y_t = sum_j w[t, j] (silu(x_t . Wg) * (x_t . Wu)) . Wd,
    e = ids[t, j] (-1: an empty slot, adds nothing), plus the shared expert's
    output: the bf16 experts of a decode step in slot order, each weight read
    once for every 32 of its expert's rows (moe_few_experts).

    x [T, H] bf16, ids [T, k] int32, w [T, k] fp32, gate_up [E*H, 2I], down
    [E*I, H], sh_gate_up [H, 2 I_s], sh_down [I_s, H] bf16; T at most 128; out
    overlaps no input."""
    return binding().few_experts(x, ids, w, gate_up, down, sh_gate_up, sh_down, out)


def layer_few(x, w_router, gate_up, down, k, bias=None, balance_bias=None, sh_gate_up=None, sh_down=None, score="softmax",
              n_groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0):
    """y [T, H] bf16, ids [T, k] int32 and w [T, k] fp32: route_logits,
    route_select and experts_few as one call (moe_few_layer)."""
    return binding().few_layer(x, w_router, gate_up, down, k, bias, balance_bias, sh_gate_up, sh_down,
                               _choice(_SCORES, score, "score"), n_groups, top_groups,
                               _choice(_GROUP_SCORES, group_score, "group_score"), bool(renorm), scale)


# ------------------------------------------------- norms around a block

def block_norm(x, weight=None, branch=None, post_weight=None, gate=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6,
               save_for_backward=False):
    """(r, h, stats): what stands between two blocks of a model, fused.

    r = residual_scale x + branch_scale gate n, with n the block's output
    branch [T, H] bf16, normed by post_weight where that is given, and
    h = rms_norm(r) weight [T, H] bf16, the next block's input.  x [T, H] (the
    residual stream) and r are fp32 or bf16; weight, post_weight [H] and gate
    [gates, H] fp32 or bf16, gates a divisor of T (a gate for every T / gates
    consecutive rows; 1: a learned scale; T: one a row).  Without branch r is
    None and h norms x; without weight h is None.  stats [2, T] fp32 with
    save_for_backward, else None, for block_norm_bwd (moe_block_norm).  As every
    operator here it records no gradients: block_norm_autograd does."""
    return binding().block_norm(x, weight, branch, post_weight, gate, residual_scale, branch_scale, eps,
                                bool(save_for_backward))


def block_norm_bwd(dh, dr, x, stats, weight=None, branch=None, post_weight=None, gate=None, residual_scale=1.0,
                   branch_scale=1.0):
    """dict(dx, d_branch, d_weight, d_post_weight, d_gate) of block_norm for
    upstream dh (of h; None without weight) and dr (of r; None: 0), each of
    its operand's type and None where the operand is.  x and branch are the
    forward's inputs (moe_block_norm_bwd)."""
    return dict(zip(("dx", "d_branch", "d_weight", "d_post_weight", "d_gate"),
                    binding().block_norm_bwd(dh, dr, stats, x, weight, branch, post_weight, gate, residual_scale,
                                             branch_scale)))


# -------------------------------------- the gradients' norm, and clipping

def grad_norm(grads):
    """The 2-norm over a list of gradients (fp32 or bf16, of any shapes, in any
    dense layout) as an fp32 scalar on the device."""
    return binding().grad_clip(grads, None, 0.0, 0.0)


def clip_grads(grads, max_norm, out=None, eps=1e-6):
    """Scales the gradients by min(1, max_norm / (norm + eps)) and returns
    their norm (grad_norm's).  In place, or into out: a list of tensors of the
    same sizes, types and strides that overlap nothing (out[i] may be grads[i])."""
    return binding().grad_clip(grads, grads if out is None else out, max_norm, eps)


def permute(ids, E, w=None):
    """counts [E], offsets [E+1], row_map [R], src_row [R] (int32), and with w
    [T,k] fp32 also w_perm [R] fp32 (the gate weight of each permuted row)."""
    _need(ids, "ids", torch.int32, 2)
    if w is not None:
        _need(w, "w", torch.float32, 2)
    T, k = ids.shape
    dev = ids.device
    nbytes = ctypes.c_size_t(0)
    call("moe_permute_workspace_size", T, k, E, ctypes.byref(nbytes))
    ws = _ws(nbytes.value, dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_map = torch.empty(T * k, dtype=torch.int32, device=dev)
    src_row = torch.empty(T * k, dtype=torch.int32, device=dev)
    w_perm = torch.empty(T * k, dtype=torch.float32, device=dev) if w is not None else None
    call("moe_permute", _p(ids), _p(w), T, k, E, _p(counts), _p(offsets), _p(row_map), _p(src_row),
         _p(w_perm), _p(ws), ws.numel(), _stream())
    if w is not None:
        return counts, offsets, row_map, src_row, w_perm
    return counts, offsets, row_map, src_row


def permute_rows(x, src_row, out=None):
    """out[r] = x[src_row[r]] for every row r (bf16 rows of width H); out: an
    existing contiguous [R, H] bf16 tensor (or row slice) to write into."""
    _need(x, "x", _BF16, 2)
    _need(src_row, "src_row", torch.int32, 1)
    R, H = src_row.shape[0], x.shape[1]
    if out is None:
        out = torch.empty((R, H), dtype=_BF16, device=x.device)
    else:
        _need(out, "out", _BF16, 2)
        if tuple(out.shape) != (R, H):
            raise ValueError("out must be [R, H]")
    call("moe_permute_rows", _p(x), _p(src_row), R, H, _p(out), _stream())
    return out


def permute_rows_scatter(x, row_map, k):
    """x_perm [T*k, H] bf16 with x_perm[row_map[t*k + j]] = x[t]: the rows of
    permute_rows(x, src_row) for the same permutation, moved token by token
    (each token row read once)."""
    _need(x, "x", _BF16, 2)
    _need(row_map, "row_map", torch.int32, 1)
    T, H = x.shape
    if row_map.shape[0] != T * k:
        raise ValueError("row_map must hold T*k entries")
    out = torch.empty((T * k, H), dtype=_BF16, device=x.device)
    call("moe_permute_rows_scatter", _p(x), _p(row_map), T, k, H, _p(out), _stream())
    return out


def sort_chunks(counts, N):
    """Rows arriving as an A x B chunk matrix in (a, b) order -> (b, a) order
    (moe_sort_chunks): src_of [N], pos_of [N] and group_offsets [B+1] (int32).
    counts: [A, B] int32 on the device, summing to N."""
    _need(counts, "counts", torch.int32, 2)
    A, B = counts.shape
    dev = counts.device
    src_of = torch.empty(N, dtype=torch.int32, device=dev)
    pos_of = torch.empty(N, dtype=torch.int32, device=dev)
    group = torch.empty(B + 1, dtype=torch.int32, device=dev)
    nbytes = ctypes.c_size_t(0)
    call("moe_sort_chunks_workspace_size", A, B, ctypes.byref(nbytes))
    ws = _ws(nbytes.value, dev)
    call("moe_sort_chunks", _p(counts), A, B, N, _p(src_of), _p(pos_of), _p(group), _p(ws), ws.numel(), _stream())
    return src_of, pos_of, group


def ep_map_replicas(ids, rep_first, rep_count, rep_list):
    """Logical expert ids [T, k] -> physical replica ids [T, k] (moe_ep_map_replicas);
    the plan tensors are int32 on the device."""
    _need(ids, "ids", torch.int32, 2)
    for t, n in ((rep_first, "rep_first"), (rep_count, "rep_count"), (rep_list, "rep_list")):
        _need(t, n, torch.int32, 1)
    T, k = ids.shape
    E, n_phys = rep_first.shape[0], rep_list.shape[0]
    out = torch.empty_like(ids)
    call("moe_ep_map_replicas", _p(ids), T, k, E, _p(rep_first), _p(rep_count), _p(rep_list), n_phys, _p(out),
         _stream())
    return out


def eplb_plan(expert_load, G, n_phys):
    """EPLB-style replication and placement on the host (moe_eplb_plan).
    expert_load: per-expert loads (sequence of ints); returns a dict of numpy
    arrays phys_to_log [n_phys], rep_first [E], rep_count [E], rep_list
    [n_phys] (int32) and rank_load [G] (int64)."""
    import numpy as np

    load = np.ascontiguousarray(np.asarray(expert_load, dtype=np.int64))
    E = load.shape[0]
    out = dict(phys_to_log=np.empty(n_phys, np.int32), rep_first=np.empty(E, np.int32),
               rep_count=np.empty(E, np.int32), rep_list=np.empty(n_phys, np.int32),
               rank_load=np.empty(G, np.int64))
    ptr = lambda a: ctypes.c_void_p(a.ctypes.data)
    call("moe_eplb_plan", ptr(load), E, G, n_phys, ptr(out["phys_to_log"]), ptr(out["rep_first"]),
         ptr(out["rep_count"]), ptr(out["rep_list"]), ptr(out["rank_load"]))
    return out


def grouped_gemm_gate_up_swiglu(x, src_row, offsets, gate_up, I, R=None, w_perm=None, save_for_backward=False):
    """h [R, I] bf16; with save_for_backward also gu_pre [R, 2I] fp32 and h_w = w_perm * h [R, I] bf16.
    src_row None: x is already in permuted order (or the dense mode when offsets is None too)."""
    _need(x, "x", _BF16, 2)
    _need(gate_up, "gate_up", _BF16, 2)
    T, H = x.shape
    E = gate_up.shape[0] // H
    if gate_up.shape != (E * H, 2 * I):
        raise ValueError("gate_up must be [E*H, 2I]")
    if src_row is not None:
        _need(src_row, "src_row", torch.int32, 1)
        R = src_row.shape[0]
    elif R is None:
        R = T
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, 1)
    if w_perm is not None:
        _need(w_perm, "w_perm", torch.float32, 1)
    h = torch.empty((R, I), dtype=_BF16, device=x.device)
    gu = hw = None
    if save_for_backward:
        if w_perm is None:
            raise ValueError("save_for_backward needs w_perm (from permute(ids, E, w))")
        gu = torch.empty((R, 2 * I), dtype=torch.float32, device=x.device)
        hw = torch.empty((R, I), dtype=_BF16, device=x.device)
    call("moe_grouped_gemm_gate_up_swiglu", _p(x), _p(src_row), _p(offsets), _p(gate_up), T, R, H, E, I,
         _p(h), _p(w_perm), _p(gu), _p(hw), _stream())
    return h, gu, hw


def grouped_gemm_down(h, offsets, down, H):
    """y_perm [R, H] bf16."""
    _need(h, "h", _BF16, 2)
    _need(down, "down", _BF16, 2)
    R, I = h.shape
    E = down.shape[0] // I
    if down.shape != (E * I, H):
        raise ValueError("down must be [E*I, H]")
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, 1)
    y = torch.empty((R, H), dtype=_BF16, device=h.device)
    call("moe_grouped_gemm_down", _p(h), _p(offsets), _p(down), R, H, E, I, _p(y), _stream())
    return y


def unpermute_combine(y_perm, row_map, w, y_shared=None, out=None):
    """y [T, H] bf16 (out: an existing contiguous [T, H] bf16 tensor or row slice to write)."""
    _need(y_perm, "y_perm", _BF16, 2)
    _need(row_map, "row_map", torch.int32, 1)
    _need(w, "w", torch.float32, 2)
    if y_shared is not None:
        _need(y_shared, "y_shared", _BF16, 2)
    T, k = w.shape
    H = y_perm.shape[1]
    if out is None:
        y = torch.empty((T, H), dtype=_BF16, device=y_perm.device)
    else:
        _need(out, "out", _BF16, 2)
        if tuple(out.shape) != (T, H):
            raise ValueError("out must be [T, H]")
        y = out
    call("moe_unpermute_combine", _p(y_perm), _p(row_map), _p(w), _p(y_shared), T, H, k, _p(y), _stream())
    return y


# ---------------------------------------------------------------- backward

def unpermute_combine_bwd(dy, src_row):
    """dy_perm [R, H] bf16: the dY row of each permuted row (unweighted, exact)."""
    _need(dy, "dy", _BF16, 2)
    _need(src_row, "src_row", torch.int32, 1)
    T, H = dy.shape
    R = src_row.shape[0]
    if (T == 0) != (R == 0) or (T > 0 and R % T):
        raise ValueError("src_row must hold T*k rows for dy [T, H]")
    k = R // T if T > 0 else 1   # an empty batch: any k >= 1 describes it
    dy_perm = torch.empty((R, H), dtype=_BF16, device=dy.device)
    call("moe_unpermute_combine_bwd", _p(dy), _p(src_row), T, H, k, _p(dy_perm), _stream())
    return dy_perm


def down_bwd_parts(I):
    n = ctypes.c_int64(0)
    call("moe_grouped_gemm_down_bwd_parts", I, ctypes.byref(n))
    return n.value


def grouped_gemm_down_bwd(dy_perm, h_w, gu_pre, w_perm, offsets, down):
    """dgu [R, 2I] bf16, d_down [E*I, H] bf16, dw_part [R, nparts] fp32."""
    _need(dy_perm, "dy_perm", _BF16, 2)
    _need(h_w, "h_w", _BF16, 2)
    _need(gu_pre, "gu_pre", torch.float32, 2)
    _need(w_perm, "w_perm", torch.float32, 1)
    _need(down, "down", _BF16, 2)
    R, I = h_w.shape
    H = dy_perm.shape[1]
    E = down.shape[0] // I
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, 1)
    dgu = torch.empty((R, 2 * I), dtype=_BF16, device=h_w.device)
    d_down = torch.empty((E * I, H), dtype=_BF16, device=h_w.device)
    parts = torch.empty((R, down_bwd_parts(I)), dtype=torch.float32, device=h_w.device)
    call("moe_grouped_gemm_down_bwd", _p(dy_perm), _p(h_w), _p(gu_pre), _p(w_perm), _p(offsets), _p(down), R,
         H, E, I, _p(dgu), _p(d_down), _p(parts), _stream())
    return dgu, d_down, parts


def route_bwd(dw_part, row_map, w, ids, E):
    """d_logits [T, E] fp32 and dw [T, k] fp32 from the per-row partials of the down backward."""
    _need(dw_part, "dw_part", torch.float32, 2)
    _need(row_map, "row_map", torch.int32, 1)
    _need(w, "w", torch.float32, 2)
    _need(ids, "ids", torch.int32, 2)
    T, k = w.shape
    dl = torch.empty((T, E), dtype=torch.float32, device=w.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=w.device)
    call("moe_route_bwd", _p(dw_part), dw_part.shape[1], _p(row_map), _p(w), _p(ids), T, E, k, _p(dl), _p(dw),
         _stream())
    return dl, dw


def grouped_gemm_gate_up_bwd(dgu, x, src_row, offsets, gate_up):
    """dx_perm [R, H] bf16, d_gate_up [E*H, 2I] bf16."""
    _need(dgu, "dgu", _BF16, 2)
    _need(x, "x", _BF16, 2)
    _need(gate_up, "gate_up", _BF16, 2)
    R, I2 = dgu.shape
    I = I2 // 2
    T, H = x.shape
    E = gate_up.shape[0] // H
    if src_row is not None:
        _need(src_row, "src_row", torch.int32, 1)
    if offsets is not None:
        _need(offsets, "offsets", torch.int32, 1)
    dx_perm = torch.empty((R, H), dtype=_BF16, device=x.device)
    d_gu = torch.empty((E * H, 2 * I), dtype=_BF16, device=x.device)
    call("moe_grouped_gemm_gate_up_bwd", _p(dgu), _p(x), _p(src_row), _p(offsets), _p(gate_up), T, R, H, E,
         I, _p(dx_perm), _p(d_gu), _stream())
    return dx_perm, d_gu


def gather_dx(dx_perm, row_map, T, k, d_logits=None, ids=None, w_router=None):
    """dX [T, H] bf16 = sum_j dx_perm[row_map] (+ d_logits . W_r^T on the chosen experts)."""
    _need(dx_perm, "dx_perm", _BF16, 2)
    _need(row_map, "row_map", torch.int32, 1)
    H = dx_perm.shape[1]
    E = 1
    ws = None
    if d_logits is not None:
        _need(d_logits, "d_logits", torch.float32, 2)
        _need(ids, "ids", torch.int32, 2)
        _need(w_router, "w_router", torch.float32, 2)
        E = w_router.shape[1]
        nbytes = ctypes.c_size_t(0)
        call("moe_gather_dx_workspace_size", H, E, ctypes.byref(nbytes))
        ws = _ws(nbytes.value, dx_perm.device)
    else:
        E = max(k, 1)
    dx = torch.empty((T, H), dtype=_BF16, device=dx_perm.device)
    call("moe_gather_dx", _p(dx_perm), _p(row_map), _p(d_logits), _p(ids), _p(w_router), T, H, E, k, _p(dx),
         _p(ws), 0 if ws is None else ws.numel(), _stream())
    return dx


def route_bwd_weight(x, d_logits):
    """d_w_router [H, E] fp32 = x^T . d_logits."""
    _need(x, "x", _BF16, 2)
    _need(d_logits, "d_logits", torch.float32, 2)
    T, H = x.shape
    E = d_logits.shape[1]
    out = torch.empty((H, E), dtype=torch.float32, device=x.device)
    call("moe_route_bwd_weight", _p(x), _p(d_logits), T, H, E, _p(out), _stream())
    return out
