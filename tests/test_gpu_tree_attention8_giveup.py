"""The bounded waits of the many-row kernel with old places, run out on purpose
(cbq_debug_tree_stall: its first block, of old places, copies nothing), as in
tests/test_gpu_tree_attention_giveup.py."""
import time

import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("old,recent,drafts,heads,kv,dim,block", [
    ([70] * 40, [9] * 40, [9] * 40, 16, 2, 128, 16),
    ([70] * 40, [9] * 40, [40] * 40, 16, 4, 128, 1),
    ([9000, 300], [20, 3], [40, 3], 16, 2, 64, 16),
    ([0] * 40, [90] * 40, [40] * 40, 16, 4, 128, 16),  # (the first block has recent places)
])
def test_wait_gives_up_and_the_next_call_is_right(torch, old, recent, drafts, heads, kv, dim, block):
    s = Setup(torch, old, recent, drafts, heads, kv, dim, block=block, seed=dim)
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
