"""The sums that the last block to arrive makes of the others' parts: the same
bits whichever block that is, with other work beside them."""
import pytest
import torch

from gpu_helpers import dev, lib
from test_gpu_few import close, make, reference

pytestmark = pytest.mark.gpu


# both products in parts; only down; only gate_up; a shared expert in parts beside routed ones that are not; many rows an expert
@pytest.mark.parametrize("shape", [(4, 1024, 4, 1, 1024, 0), (9, 256, 8, 2, 2048, 0), (2, 4096, 8, 2, 64, 0), (70, 1024, 4, 1, 64, 3200), (16, 2048, 32, 8, 768, 768),
                                   (128, 512, 4, 2, 256, 0)], ids=str)
def test_the_same_bits_again(shape):
    moe = lib()
    a = make(*shape)
    want = moe.experts_few(*a)
    close(want, reference(*a))
    square = torch.ones((2048, 2048), dtype=torch.bfloat16, device=dev())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 2]):
            if i % 3 == 0:
                square @ square
            got.append(moe.experts_few(*a))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    moe.sync_status()


def test_an_out_that_overlaps_an_input_is_refused():
    """Tokens' outputs are written while other tokens' inputs are still read."""
    moe = lib()
    x, ids, w, gu, dn, sgu, sdn = make(6, 128, 8, 2, 64, 64)
    buffer = torch.zeros((12, 128), dtype=torch.bfloat16, device=dev())
    buffer[:6] = x
    rows = buffer[:6]
    for bad in ((rows, rows), (rows, buffer[1:7]), (rows, buffer[5:11]), (x, gu.view(-1, 128)[3:9]), (x, dn[:6]), (x, sdn[58:64]), (x, sgu.view(-1, 128)[:6])):
        with pytest.raises(ValueError, match="overlaps"):
            moe.experts_few(bad[0], ids, w, gu, dn, sgu, sdn, out=bad[1])
    assert torch.equal(rows, x)
    y = moe.experts_few(rows, ids, w, gu, dn, sgu, sdn, out=buffer[6:])      # beside it
    assert torch.equal(y, moe.experts_few(x, ids, w, gu, dn, sgu, sdn)) and torch.equal(rows, x)
    moe.sync_status()
