"""Distributions and drawn tokens in the free columns of the logits' own tensor:
the same as in tensors of their own."""
import pytest

from tests.gpu_util import cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("n", [1, 5, 200])
@pytest.mark.parametrize("V", [7, 1001, 32000])
def test_halves_of_rows(torch, n, V):
    g = torch.Generator(device="cuda").manual_seed(n + V)
    both = torch.randn((n, 2 * V + 3), generator=g, device="cuda")
    u, p = torch.rand((n,), generator=g, device="cuda"), torch.rand((n,), generator=g, device="cuda")
    kept = both.clone()
    want, ids = cbq.cbq_probs(both[:, :V].contiguous(), None, None, p, None, u)
    out, got = cbq.cbq_probs(both[:, :V], None, None, p, None, u, out=both[:, V:2 * V])
    assert torch.equal(out, want) and torch.equal(got, ids)
    assert torch.equal(both[:, :V], kept[:, :V]) and torch.equal(both[:, 2 * V:], kept[:, 2 * V:])
    back = cbq.cbq_probs(kept[:, V + 3:], None, None, p, None, out=kept[:, :V])  # the other way round
    assert torch.equal(back, cbq.cbq_probs(kept[:, V + 3:].contiguous(), None, None, p, None))
    with pytest.raises(cbq.CbqError):
        cbq.cbq_probs(kept[:, :V], None, None, p, None, out=kept[:, V - 1:2 * V - 1])
