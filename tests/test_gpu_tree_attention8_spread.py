"""Values' scales at both ends of their range in one row, neighbouring blocks
and different chunks, either end first: the sum of the weights, which has no
scale in it, is the same whatever the scales (the lse shows it alone), and the
result keeps the large ones' share of it.  Tolerances as in
test_gpu_tree_attention8.py."""
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup

pytestmark = pytest.mark.gpu

# old, recent, drafts, heads, kv heads, head size, block of a scale
PATHS = {"a warp a row": ([100], [9], [3], 4, 2, 80, 16), "one block": ([60], [0], [3], 4, 2, 64, 4),
         "a cluster": ([300, 40], [20, 3], [1, 2], 16, 8, 128, 16), "heads of 256": ([700], [30], [5], 6, 2, 256, 16),
         "parts": ([8192], [100], [2], 16, 8, 128, 16), "parts, a token a scale": ([8192], [100], [1], 16, 8, 64, 1),
         "64 rows": ([300], [5], [20], 3, 1, 64, 16), "many rows": ([600, 50], [9, 0], [40, 7], 2, 2, 128, 16),
         "many rows, two row tiles": ([600], [9], [64], 16, 2, 128, 16),
         "many rows, 4 tokens a scale": ([600], [9], [40], 2, 2, 128, 4),
         "many rows, parts": ([6000], [50], [40], 2, 1, 128, 16),
         "many rows, parts, 4 tokens a scale": ([6000], [50], [40], 2, 1, 128, 4),
         "many rows, heads of 64": ([5000, 300], [20, 1], [40, 3], 4, 2, 64, 16)}


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _scales(torch, s, exponent):
    """Every block's value scale is 2^exponent(place of its first token, places of the sequence)."""
    e = torch.zeros((s.vs.shape[0], s.vs.shape[1]))
    for i, n in enumerate(s.old):
        for p in range(0, int(n), s.block):
            e[int(s.table8[i][p // s.page8]), p % s.page8 // s.block] = exponent(p, int(n))
    s.vs = torch.exp2(e).cuda()[..., None].expand(s.vs.shape).contiguous()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("ends", [(-20, 110), (-80, 112), (-80, 50), (0, 112)])
def test_both_ends(torch, path, ends):
    old, recent, drafts, heads, kv, dim, block = PATHS[path]
    small, large = ends
    orders = {"small ones first": lambda p, n: small if p < n // 2 else large,
              "large ones first": lambda p, n: large if p < n // 2 else small,
              "in turn": lambda p, n: (small, large)[p // block % 2],
              "one large, the last": lambda p, n: large if p + block >= n else small,
              "one large, the first": lambda p, n: large if p == 0 else small,
              "up by steps": lambda p, n: small + (large - small) * p // n}
    sharp = 3.0 if ends == (-80, 112) else 0.02  # scores far apart, too
    for seed, (name, exponent) in enumerate(orders.items()):
        s = Setup(torch, old, recent, drafts, heads, kv, dim, 16, 16, block, seed=seed, sharp=sharp)
        _scales(torch, s, exponent)
        out, lse = s.run(out=torch.empty(s.q.shape, device="cuda"))
        try:
            s.check(out, lse)
        except AssertionError as e:
            raise AssertionError(name) from e


@pytest.mark.parametrize("path", ["a cluster", "parts", "many rows", "many rows, parts", "many rows, 4 tokens a scale"])
def test_scores_do_not_hang_on_the_values_scales(torch, path):
    """The same keys under scales of every size: lse within its tolerance of that under scales of 1."""
    old, recent, drafts, heads, kv, dim, block = PATHS[path]
    s = Setup(torch, old, recent, drafts, heads, kv, dim, 16, 16, block, "float16", seed=4, sharp=0.5)
    for exponent in (lambda p, n: 0, lambda p, n: (p * 37 // block) % 193 - 80, lambda p, n: 112 - 192 * p // n):
        _scales(torch, s, exponent)
        out, lse = s.run(out=torch.empty(s.q.shape, device="cuda"))
        s.check(out, lse)
