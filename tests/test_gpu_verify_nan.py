"""NaN in the rows that the verification reads (cbq_verify) counts as 0: the
target's and the drafter's, at a child's token and elsewhere, and whole rows of
it.  The answers are those of the definition in 64 bits on rows with 0 in the
NaNs' place; what is below 0 counts as 0 too.  A given number u of NaN accepts
nothing."""
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
    none = lambda x: np.where(x > 0, x, 0.0)  # noqa: E731
    p, q = (None if x is None else none(x.double().cpu().numpy()) for x in (c["p"], c["q"]))
    compared = 0
    for s in range(len(c["start"]) - 1):
        a, b = c["start"][s], c["start"][s + 1]
        want, token, margin = behind_ref.verify(p[a:b], None if q is None else q[a:b], c["tokens"][a:b], c["parent"][a:b],
                                                c["u"][a:b], c["un"][s])
        if margin >= 2.0 ** -40:
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


def test_below_zero(torch):
    """A row with numbers below 0 among its tokens, the children's too."""
    for kind in ("chain", "star"):
        c = _case(torch, [5, 9, 2], 700, 7, kind, near=2.0)
        for k, n in (("p", 3), ("q", 5)):
            c[k][:, ::n] *= -1
        for row, token in list(_children(c))[::3]:
            c["q"][row, token] = -0.5
        _check(torch, c, 9)


@pytest.mark.parametrize("drawn", [True, False])
def test_given_numbers(torch, drawn):
    """u NaN accepts nothing, u_next NaN draws the first token with any weight left."""
    c = _case(torch, [2, 2, 2], 400, 6, "chain", drawn)
    c["u"][:] = float("nan")
    c["un"][:] = float("nan")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    _, count, nxt = cbq.cbq_verify(c["p"], c["q"], dev(c["tokens"]), dev(c["parent"]), dev(c["start"]), dev(c["u"]), dev(c["un"]), max_tok=2)
    assert count.tolist() == [1, 1, 1]
    for s in range(3):
        r = c["p"][2 * s].double()
        if drawn:
            r = r - c["q"][2 * s].double()
        else:
            r[int(c["tokens"][2 * s + 1])] = 0
        assert int(nxt[s]) == int((r > 0).nonzero()[0])
