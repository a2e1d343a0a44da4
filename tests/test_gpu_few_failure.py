"""The bounded waits of the few-token experts: with no weights arriving
(the test hook) the launch ends by itself, the timeout is reported, the
context stays usable and the next call is right."""
import time

import pytest
import torch

from gpu_helpers import lib
from test_gpu_few import close, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", ((1, 2048, 16, 8, 768, 0), (40, 512, 8, 2, 256, 128)), ids=str)
def test_a_stalled_producer_is_reported(shape):
    moe = lib()
    T, H, E, k, I, I_s = shape
    a = make(T, H, E, k, I, I_s)
    want = reference(*a)
    L = moe.load()
    moe.set_wait_limit_ns(20_000_000)
    L.moe_test_stall_gemm_producer(1)
    try:
        t0 = time.time()
        moe.experts_few(*a)
        with pytest.raises(moe.MoEError, match="MOE_ERR_TIMEOUT"):
            moe.sync_status()
        assert time.time() - t0 < 5.0
    finally:
        L.moe_test_stall_gemm_producer(0)
        moe.set_wait_limit_ns(0)
    y = moe.experts_few(*a)
    moe.sync_status()
    close(y, want)
