"""Factors on the scores beyond what fp32 holds: a large query, small key scales
that make up for it, and among them keys of nothing but zeros under the largest
scale, whose scores are 0.  Tolerances as in test_gpu_tree_attention8.py."""
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup
from tests.test_gpu_tree_attention8_spread import PATHS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("path", PATHS)
def test_zeros_under_a_large_scale(torch, path):
    old, recent, drafts, heads, kv, dim, block = PATHS[path]
    s = Setup(torch, old, recent, drafts, heads, kv, dim, 16, 16, block, seed=3)
    s.q = (s.q.float() * 2.0 ** 60).bfloat16()
    s.kc.zero_()
    s.ks = torch.full_like(s.ks, 2.0 ** -39)
    for i, n in enumerate(s.old):  # every third block of 16 places
        for p in range(0, int(n), 48):
            page = int(s.table8[i][p // s.page8])
            s.k8[page].view(torch.uint8).zero_()
            s.ks[page] = 2.0 ** 112
    out, lse = s.run(scale=2.0 ** -28)
    assert bool(torch.isfinite(out).all())
    s.check(out, lse, 2.0 ** -28)
