"""Heads of 256 over long contexts: keys that go round the ring of tiles,
split over blocks and joined by the second kernel, for each number of rows a
block; against the definition in 64 bits, with test_gpu_tree_attention's
tolerances."""
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention import Setup, _go
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _room(s):
    total, heads, dim = s.q.shape
    return cbq.cbq_tree_attention_workspace(len(s.ctx), total, s.max_tok, s.max_len, heads, s.kc.shape[2], dim)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("ctx,drafts,heads,kv", [
    ([5000], [3], 8, 2),             # 12 rows, parts joined by eight warps a row
    ([5000], [5], 20, 4),            # 25 rows
    ([5000], [13], 4, 1),            # 52 rows
    ([3000], [40], 4, 1),            # three tiles of rows
    ([1500] * 20, [5] * 20, 32, 8),  # 3,200 rows
])
def test_long(torch, dtype, ctx, drafts, heads, kv):
    s = _go(torch, ctx, drafts, heads, kv, 256, 48, dtype=dtype, seed=ctx[0] + drafts[0])
    assert _room(s) > 16, "meant for the second kernel"


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_long_in_a_cluster(torch, dtype):
    """Few blocks of many keys each; sequences that end in the first one, and one without context."""
    s = _go(torch, [9000, 0, 77], [33, 5, 64], 8, 4, 256, 48, dtype=dtype, seed=9)
    assert _room(s) == 16


@pytest.mark.parametrize("n", [191, 192, 193, 255, 256, 257, 1023, 1025])
def test_lengths(torch, n):
    """Around the borders of tiles and of the ring, with pages that end inside a tile."""
    _go(torch, [n], [5], 4, 2, 256, 5, seed=n)
    _go(torch, [n, 900, 3], [20, 1, 8], 4, 2, 256, 32, seed=n, dtype="float16")


def test_moving_top_repeats_and_output_type(torch):
    s = Setup(torch, [4000], [9], 4, 1, 256, 16, seed=7)
    assert _room(s) > 16
    order = torch.from_numpy(s.table[0].astype("int64")).cuda()
    s.kc[order] *= torch.linspace(0.01, 3.0, len(order), device="cuda").to(s.dt)[:, None, None, None]
    out, lse = s.run()
    s.check(out, lse)
    for _ in range(3):
        again, lse2 = s.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    f = torch.empty(out.shape, dtype=torch.float32, device="cuda")
    s.run(out=f)
    assert torch.equal(f.to(s.dt), out)


def test_bad_page_in_a_long_context(torch):
    """A page outside the cache is reported, not seen, and nothing else changes."""
    s = Setup(torch, [3000], [3], 4, 2, 256, 16, seed=8)
    keep = s.table.copy()
    s.table[0, 100] = s.kc.shape[0]
    out, lse = s.run()
    assert s.err.item() == cbq.CBQ_DEVERR_BAD_SLOT
    s.table = keep[:, [i for i in range(keep.shape[1]) if i != 100]]
    s.ctx = s.ctx - 16
    s.check(out, lse)
