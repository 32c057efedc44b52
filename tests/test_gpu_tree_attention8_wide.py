"""Many rows over old places in 8 bits: pages and blocks of scales that are whole
sixteens of tokens, and others, have kernels of their own; both over the range
of the scales, beside one another, and where places end inside a tile."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup, _go

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("page8,block", [(16, 16), (48, 16), (128, 64), (24, 24), (16, 8)])
@pytest.mark.parametrize("drafts,heads,kv,dim", [(40, 8, 2, 128), (64, 8, 1, 64), (33, 4, 1, 128)])
def test_pages(torch, page8, block, drafts, heads, kv, dim):
    for old, recent in (([700, 1, 63, 0], [5, 0, 64, 3]), ([3000], [1])):
        n = len(old)
        _go(torch, old, recent, [drafts] + [7] * (n - 1), heads, kv, dim, 16, page8, block, seed=page8 + dim, spread=6)


@pytest.mark.parametrize("block", [16, 4])
@pytest.mark.parametrize("e", [-80, 112])
def test_ends_of_the_scales(torch, block, e):
    """All values tiny or huge: results in fp32, relative to their size."""
    s = Setup(torch, [500], [0], [40], 4, 2, 128, 16, 16, block, seed=e + 80)
    s.vs = torch.full_like(s.vs, 2.0 ** e)
    out, lse = s.run(out=torch.empty(s.q.shape, device="cuda"), max_new=40)
    s.kc.zero_(), s.vc.zero_()
    own = s.mask.copy()
    s.mask[:] = 0  # (the drafts' own values are of ordinary size: none is seen)
    out, lse = s.run(out=torch.empty(s.q.shape, device="cuda"))
    s.check(out, lse)
    assert float(out.abs().max()) > 2.0 ** e and own.any()


@pytest.mark.parametrize("block", [16, 4])
def test_scales_far_apart(torch, block):
    """Neighbouring blocks' values 2^40 apart, with scores that make up for it or not."""
    for seed, sharp in ((1, 0.01), (2, 4.0)):
        s = Setup(torch, [900], [20], [40], 8, 2, 128, 16, 32, block, seed=seed, spread=20, sharp=sharp)
        out, lse = s.run()
        s.check(out, lse)
        assert int(s.err) == 0 and np.isfinite(out.float().cpu().numpy()).all()
