"""NaN counts as 0 in everything that the verification reads (cbq_verify):
target's and drafter's rows, at a child's token and elsewhere, whole rows of
them, and the given numbers.  The answers are those of the definition in 64 bits
on the inputs with 0 in the NaNs' place."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import cuda
from tests.test_gpu_verify import _case
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _check(torch, c, max_tok):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    path, count, nxt = cbq.cbq_verify(c["p"], c["q"], dev(c["tokens"]), dev(c["parent"]), dev(c["start"]), dev(c["u"]),
                                      dev(c["un"]), max_tok=max_tok)
    none = lambda x: np.where(np.isnan(x), 0.0, x)  # noqa: E731
    p, q = (None if x is None else none(x.double().cpu().numpy()) for x in (c["p"], c["q"]))
    compared = 0
    for s in range(len(c["start"]) - 1):
        a, b = c["start"][s], c["start"][s + 1]
        want, token, margin = behind_ref.verify(p[a:b], None if q is None else q[a:b], c["tokens"][a:b], c["parent"][a:b],
                                                none(c["u"][a:b]), none(c["un"][s:s + 1])[0])
        if margin >= 2.0 ** -40 or np.isnan(c["u"][a:b]).any() or np.isnan(c["un"][s]):  # (a given 0 is exact)
            assert (path[s].tolist(), int(count[s]), int(nxt[s])) == (want + [-1] * (max_tok - len(want)), len(want), token), s
            compared += 1
    assert compared >= len(c["start"]) - 2
    return path, count, nxt


def _children(c):
    """(row of the parent, token) of every child."""
    for s in range(len(c["start"]) - 1):
        for i in range(c["start"][s] + 1, c["start"][s + 1]):
            yield int(c["start"][s] + c["parent"][i]), int(c["tokens"][i])


@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("V", [8, 517, 4099])
@pytest.mark.parametrize("where", ["p", "q"])
def test_at_the_childrens_tokens(torch, kind, V, where):
    for drawn in (True, False):
        for u in (0.0, 0.5, 1.0 - 2.0 ** -24):
            c = _case(torch, [5, 9, 2], V, V, kind, drawn, near=2.0)
            c["u"][:] = u
            for row, token in list(_children(c))[::2]:
                if c[where] is not None:
                    c[where][row, token] = float("nan")
            _check(torch, c, 9)


@pytest.mark.parametrize("V", [9, 1003, 129280])
@pytest.mark.parametrize("where", ["p", "q", "both"])
def test_elsewhere(torch, V, where):
    """Every third of the tokens, the children's not among them: passes over the rows and the draw."""
    for kind in ("chain", "star"):
        for near in (0.7, 3.0):
            c = _case(torch, [5, 9, 2], V, 3, kind, near=near)
            kept = {k: c[k].clone() for k in "pq"}
            for k in "pq":
                if where in (k, "both"):
                    c[k][:, ::3] = float("nan")
                    for row, token in _children(c):
                        c[k][row, token] = kept[k][row, token]
            _check(torch, c, 9)


def test_whole_rows(torch):
    """A drafter's row of nothing but NaN has no weight: its children are accepted where the target has any."""
    c = _case(torch, [4, 4, 4], 300, 5, "star")
    c["q"][0] = float("nan")
    c["p"][4] = float("nan")
    c["p"][8] = c["q"][8] = float("nan")
    c["u"][:] = 0.99
    _, count, nxt = _check(torch, c, 4)
    assert count.tolist() == [2, 1, 1] and nxt.tolist()[1:] == [-1, -1]


@pytest.mark.parametrize("drawn", [True, False])
def test_given_numbers(torch, drawn):
    """u NaN accepts what has any weight, u_next NaN draws the first token with any."""
    c = _case(torch, [5, 6, 3], 400, 6, "chain", drawn)
    c["u"][:] = float("nan")
    c["un"][:] = float("nan")
    _, count, nxt = _check(torch, c, 6)
    assert count.tolist() == [5, 6, 3] and nxt.tolist() == [0, 0, 0]
