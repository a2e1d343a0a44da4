"""The bounded waits of the norms around a block: with no rows of x arriving
(the test hook) a launch ends by itself, the timeout is reported, the context
stays usable and the next call is right."""
import time

import pytest
import torch

from gpu_helpers import lib
from test_gpu_block_norm import EPS, inputs, run_both

pytestmark = pytest.mark.gpu

# rows enough for a ring to be filled more than once and not to be; one warp a row, and many; dr in the
# ring and beside it; every kind of gate; sums over columns through the ring's memory
CASES = [dict(T=1, H=64), dict(T=3000, H=256, post="f32", gates=1), dict(T=3000, H=2048, x="f32", post="f32"), dict(T=700, H=7168, x="f32", post="f32", gates=1),
         dict(T=640, H=512, gates=4, post="f32"), dict(T=640, H=4096, x="f32", gates=640, post="f32"), dict(T=500, H=1024, weight=None),
         dict(T=500, H=1024, branch=False)]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_rows_that_do_not_arrive_are_reported(kw):
    moe = lib()
    d, up = inputs(**kw)
    how = dict(weight=d["weight"], branch=d["branch"], post_weight=d["post_weight"], gate=d["gate"])
    stats = moe.block_norm(d["x"], eps=EPS, save_for_backward=True, **how)[2]
    torch.cuda.synchronize()
    moe.set_wait_limit_ns(20_000_000)
    try:
        for call in (lambda: moe.block_norm(d["x"], eps=EPS, **how), lambda: moe.block_norm_bwd(up["dh"], up["dr"], d["x"], stats, **how)):
            moe._lib.call("moe_test_stall_gemm_producer", 1)
            t0 = time.time()
            call()
            moe._lib.call("moe_test_stall_gemm_producer", 0)
            with pytest.raises(moe.MoEError, match="MOE_ERR_TIMEOUT"):
                moe.sync_status()
            assert time.time() - t0 < 5.0
    finally:
        moe._lib.call("moe_test_stall_gemm_producer", 0)
        moe.set_wait_limit_ns(0)
    run_both(moe, d, up)
