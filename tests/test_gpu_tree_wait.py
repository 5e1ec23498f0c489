"""Failure detection of the tree attention, without a fault: a wait for tiles that runs out.

Under a limit of 1 ns the warps only poll, a few times in well under a microsecond, while the tiles come
from memory that the L2 does not hold: the first waits give up, and every warp waits (with a limit) for
its own copies and products in flight and leaves.  The call is then over, the status is a timeout, and
under the default limit the next call in the same context is right."""
import pytest
import torch

from test_gpu_append import swa  # noqa: F401  (the fixture)
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

SWIATTN_ETIMEOUT = 4


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,d", [(64, 128), (4, 64)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(swa, page, d, kind):
    c = Case([40, 9], [3000, 2500], 4, 2, d, page, kind, 1000, routed=0.5, seed=31)
    want = c.run(swa)
    assert swa.get_device_error() == 0
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()   # larger than the L2
    swa.set_wait_limit_ns(1)
    try:
        c.run(swa)
        torch.cuda.synchronize()
        assert swa.get_device_error() == SWIATTN_ETIMEOUT
    finally:
        swa.set_wait_limit_ns(0)
    got = c.run(swa)
    assert swa.get_device_error() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)
