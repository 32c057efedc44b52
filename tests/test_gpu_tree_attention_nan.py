"""A query with NaN: its row of the result and its lse are NaN, however the
keys are split and joined, and no other row changes by a bit.  (A row that sees
nothing gives zeros and -inf: that is no answer to a NaN of the layer before.)"""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention import Setup
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


# ctx, drafts, heads, kv heads, head size, whether parts go to a second kernel; named by what takes the keys
PATHS = {
    "a warp a row": ([200], [3], 4, 2, 80, False),
    "one block": ([60], [3], 4, 2, 64, False),
    "one block, 64 rows": ([60], [20], 3, 1, 64, False),
    "a cluster": ([300], [1], 32, 8, 128, False),
    "a cluster, heads of 256": ([250], [5], 6, 2, 256, False),
    "parts, eight warps a row": ([8191], [5], 32, 8, 128, True),
    "parts, a warp a row": ([2000] * 24, [5] * 24, 32, 8, 128, True),
    "many rows, one block": ([70] * 40, [9] * 40, 16, 2, 128, False),
    "many rows, one block, both groups": ([70] * 40, [40] * 40, 16, 4, 128, False),
    "many rows, parts": ([3000], [40], 8, 1, 128, True),
    "many rows, parts, heads of 64": ([9000, 300], [40, 3], 16, 2, 64, True),
}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("where", ["one value", "all values"])
def test_nan_query(torch, path, dtype, where):
    ctx, drafts, heads, kv, dim, parts = PATHS[path]
    s = Setup(torch, ctx, drafts, heads, kv, dim, 16, dtype=dtype, seed=dim)
    room = cbq.cbq_tree_attention_workspace(len(ctx), int(s.start[-1]), s.max_tok, s.max_len, heads, kv, dim)
    assert (room > 16) == parts, "another path than the one meant"
    whole, lse = s.run()
    row, head = len(s.mask) - 1, heads - 1
    s.q[row, head, 7:8 if where == "one value" else None] = float("nan")
    s.q[0, 0] = float("nan")
    out, lse2 = s.run()
    odd = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    odd[row, head] = odd[0, 0] = True
    assert torch.isnan(out[odd]).all(), "the result hides it"
    assert torch.isnan(lse2[odd]).all(), "the lse hides it"
    assert torch.equal(out[~odd], whole[~odd]) and torch.equal(lse2[~odd], lse[~odd])
    assert s.err.item() == 0


@pytest.mark.parametrize("path", PATHS)
def test_nan_keys(torch, path):
    """A committed key with NaN, alone in its part of the keys or not, is every row's."""
    ctx, drafts, heads, kv, dim, _ = PATHS[path]
    s = Setup(torch, ctx, drafts, heads, kv, dim, 16, seed=dim)
    i = len(ctx) - 1  # one kv head of the last sequence
    p = s.ctx[i] - 1
    s.kc[int(s.table[i][p // 16]), int(p % 16), kv - 1, 3] = float("nan")
    out, lse = s.run()
    rows = slice(int(s.start[i]), int(s.start[i + 1]))
    h = slice((kv - 1) * (heads // kv), heads)
    assert torch.isnan(out[rows, h]).all() and torch.isnan(lse[rows, h]).all()
    rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    rest[rows, h] = False
    assert torch.isfinite(out[rest]).all() and torch.isfinite(lse[rest]).all()


def test_nan_key_alone_in_a_part(torch):
    """The last part of a split row holds one key, whose score is NaN."""
    for ctx, drafts, heads, kv, dim in (([8192], [1], 8, 8, 128), ([12288], [33], 8, 1, 128)):
        s = Setup(torch, ctx, drafts, heads, kv, dim, 64, seed=5)
        for p in range(s.ctx[0] - 300, s.ctx[0] + drafts[0]):
            s.kc[int(s.table[0][p // 64]), int(p % 64)] = float("nan")
        out, lse = s.run()
        assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_nothing_seen_is_still_zeros(torch):
    """Beside a NaN row in every path: rows that see nothing keep zeros and -inf."""
    for path, (ctx, drafts, heads, kv, dim, _) in PATHS.items():
        ctx = [0] + ctx
        s = Setup(torch, ctx, [3] + drafts, heads, kv, dim, 16, seed=1)
        s.mask[:3] = 0
        s.q[3] = float("nan")
        out, lse = s.run()
        assert not out[:3].any() and np.isneginf(lse[:3].cpu().numpy()).all(), path
        assert torch.isnan(out[3]).all() and torch.isnan(lse[3]).all(), path
