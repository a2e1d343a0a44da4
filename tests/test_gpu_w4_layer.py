"""moe_forward_w4 at batches of more rows per expert than its limit for the
bf16 grouped GEMMs, with and without it."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_routing_layer import layer_inputs

pytestmark = pytest.mark.gpu

H, E, K_TOKEN, I, I_SHARED = 256, 8, 2, 128, 192


def layer(moe, T):
    d, s = layer_inputs(T, T, H, E, I), layer_inputs(T + 1, T, H, 1, I_SHARED)
    return (d, moe.W4Experts.quantize(d["gate_up"], d["down"], E, 64),
            moe.W4Experts.quantize(s["gate_up"], s["down"], 1, 64, zeros=True))


def test_a_token_of_the_layer_does_not_depend_on_the_batch():
    """100 rows per expert and 400 of the shared one: each token's bits are
    those that it has alone, or among few."""
    moe = lib()
    T = 400
    d, experts, shared = layer(moe, T)
    routing = moe.Routing(score="sigmoid", n_groups=4, top_groups=2)
    kw = dict(shared=shared, routing=routing, balance_bias=d["bias"])
    y, ids, w = moe.moe_forward_w4(d["x"], d["wr"], experts, K_TOKEN, **kw)
    for a, b in ((0, 1), (5, 12), (100, 164), (399, 400)):
        yp, idp, wp = moe.moe_forward_w4(d["x"][a:b].contiguous(), d["wr"], experts, K_TOKEN, **kw)
        assert torch.equal(idp, ids[a:b]) and torch.equal(wp, w[a:b]) and torch.equal(yp, y[a:b])
    moe.sync_status()


@pytest.mark.parametrize("T", (13, 110, 400))
def test_bf16_rows_of_routed_experts(T):
    """With a limit of 48 rows per expert, which 400 tokens pass: bit for bit
    the 4-bit kernels, or moe_forward on the decoded weights."""
    moe = lib()
    d, experts, _ = layer(moe, T)
    limit = moe.layer.W4_MAX_ROWS_PER_EXPERT
    y, ids, w = moe.moe_forward_w4(d["x"], d["wr"], experts, K_TOKEN, bf16_rows=limit)
    if T * K_TOKEN > limit * E:
        want, _ = moe.moe_forward(d["x"], d["wr"], *experts.dequantize(), K_TOKEN)
    else:
        want = moe.w4_down_combine(moe.w4_gate_up_swiglu(d["x"], ids, *experts.gate_up), ids, w, *experts.down)
    assert torch.equal(y, want)
    g = moe.DecodeGraph(T, d["wr"], experts, K_TOKEN, bf16_rows=limit)
    assert torch.equal(g(d["x"]), y)
    moe.sync_status()


@pytest.mark.parametrize("T", (13, 110, 400))
def test_bf16_rows(T):
    """With a limit of 48 rows per expert: 13 tokens stay under it, at 110 the
    shared expert's rows pass twice that, at 400 all do; either side is, bit for bit,
    the 4-bit kernels or moe_forward on the decoded weights."""
    moe = lib()
    d, experts, shared = layer(moe, T)
    limit = moe.layer.W4_MAX_ROWS_PER_EXPERT
    y, ids, w = moe.moe_forward_w4(d["x"], d["wr"], experts, K_TOKEN, shared=shared, bf16_rows=limit)
    sh_gate_up, sh_down = shared.dequantize()
    if T * K_TOKEN > limit * E:
        want, st = moe.moe_forward(d["x"], d["wr"], *experts.dequantize(), K_TOKEN, sh_gate_up=sh_gate_up, sh_down=sh_down)
        assert torch.equal(ids, st.ids) and torch.equal(w, st.w)
    else:
        if T > 2 * limit:
            hs, _, _ = moe.grouped_gemm_gate_up_swiglu(d["x"], None, None, sh_gate_up, I_SHARED)
            ys = moe.grouped_gemm_down(hs, None, sh_down, H)
        else:
            ys = moe.w4_down_combine(moe.w4_gate_up_swiglu(d["x"], None, *shared.gate_up), None, None, *shared.down)
        h = moe.w4_gate_up_swiglu(d["x"], ids, *experts.gate_up)
        want = moe.w4_down_combine(h, ids, w, *experts.down, y_shared=ys)
    assert torch.equal(y, want)
    g = moe.DecodeGraph(T, d["wr"], experts, K_TOKEN, shared=shared, bf16_rows=limit)
    assert torch.equal(g(d["x"]), y)
    moe.sync_status()


def test_memory_of_the_decoded_weights():
    """gate_up's bf16 weights are released before down's are made: the call's
    peak stays under the two together."""
    moe = lib()
    T, H_, E_, I_ = 512, 1024, 64, 512
    g = torch.Generator(device=dev()).manual_seed(1)
    bf = lambda *s: (0.03 * torch.randn(s, generator=g, device=dev())).bfloat16()
    gate_up, down = bf(E_ * H_, 2 * I_), bf(E_ * I_, H_)
    both = (gate_up.numel() + down.numel()) * 2
    experts = moe.W4Experts.quantize(gate_up, down, E_)
    del gate_up, down
    x, wr = bf(T, H_), bf(H_, E_).float()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    moe.moe_forward_w4(x, wr, experts, 8, bf16_rows=0)
    moe.sync_status()
    rows = T * 8
    activations = 2 * (2 * rows * H_ + rows * I_ + 2 * T * H_) + 4 * T * E_ + (8 << 20)
    assert torch.cuda.max_memory_allocated() - before < both * 2 // 3 + activations < both + activations
