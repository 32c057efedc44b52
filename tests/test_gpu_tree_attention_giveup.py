"""The bounded waits of the tree attention's many-row kernel, run out on
purpose (cbq_debug_tree_stall: its first block copies nothing).  The call
returns, sets the timeout bit alone and leaves every other block's rows as they
are; the next calls give the bits of a call before.  No GPU fault is involved:
the waits end by their limit."""
import time

import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention import Setup
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("ctx,drafts,heads,kv,dim", [
    ([70] * 40, [9] * 40, 16, 2, 128),     # a block a row tile: the groups share out the keys
    ([70] * 40, [40] * 40, 16, 4, 128),    # both groups with rows of their own
    ([9000, 300], [40, 3], 16, 2, 64),     # parts, joined by the second kernel
    ([9000, 300], [16, 3], 16, 2, 128),
])
def test_wait_gives_up_and_the_next_call_is_right(torch, ctx, drafts, heads, kv, dim):
    s = Setup(torch, ctx, drafts, heads, kv, dim, 16, seed=dim)
    whole, lse = s.run()
    assert s.err.item() == 0
    cbq.cbq_debug_tree_stall(1)
    try:
        t0 = time.monotonic()
        out, lse2 = s.run()
        torch.cuda.synchronize()
        took = time.monotonic() - t0
    finally:
        cbq.cbq_debug_tree_stall(0)
    assert s.err.item() == cbq.CBQ_DEVERR_PIPE_TIMEOUT, f"error word {s.err.item():#x}"
    assert 0.5 < took < 10, "another kernel than the one meant, or waits without a limit"
    rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    rest[:drafts[0], :heads // kv] = False
    assert torch.equal(out[rest], whole[rest]) and torch.equal(lse2[rest], lse[rest])
    s.err.zero_()
    for _ in range(2):
        out, lse2 = s.run()
        assert torch.equal(out, whole) and torch.equal(lse2, lse)
    assert s.err.item() == 0


def test_other_kernels_are_not_touched(torch):
    s = Setup(torch, [300], [3], 8, 2, 128, 16)
    whole, lse = s.run()
    cbq.cbq_debug_tree_stall(1)
    try:
        out, lse2 = s.run()
        torch.cuda.synchronize()
    finally:
        cbq.cbq_debug_tree_stall(0)
    assert s.err.item() == 0 and torch.equal(out, whole) and torch.equal(lse2, lse)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_debug_tree_stall(2)
