"""Rows of inputs and outputs that lie in turn in one tensor share no byte and
are taken; where a row of one meets a row of the other they are refused (CPU
only: pointers alone, and no GPU is touched)."""
import ctypes

import pytest

from verify_matvec_gb300 import build, cbq

P = ctypes.c_void_p
AT = 0x100000


@pytest.fixture(scope="module")
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    build.build()
    return cbq.load()


def _probs(lib, x, out, n, V, xs, os, ids=None, u=None):
    return lib.cbq_probs(P(x), 0, n, V, xs, None, None, None, None, P(u) if u else None, P(out), os, P(ids) if ids else None, None)


def _taken(rc):
    return rc not in (cbq.CBQ_OK, cbq.CBQ_EINVAL)  # (it gets to the check for a GPU)


@pytest.mark.parametrize("n", [1, 2, 5, 256])
def test_halves_of_rows(lib, n):
    V = 10
    for st in (20, 23, 24):
        for shift in range(-2, 3):  # (n rows of V, so many rows apart)
            assert _taken(_probs(lib, AT, AT + (V + shift * st) * 4, n, V, st, st))
            assert _taken(_probs(lib, AT + (V + shift * st) * 4, AT, n, V, st, st))
    st = 23  # three free columns: out may begin in V .. V + 3 of the row
    for off in range(-3 * st, 3 * st):
        meets = any(abs(off + k * st) < V for k in range(-(n - 1), n))
        rc = _probs(lib, AT, AT + off * 4, n, V, st, st)
        assert _taken(rc) if not meets else rc == cbq.CBQ_EINVAL, off


@pytest.mark.parametrize("na,sa,nb,sb", [(4, 23, 4, 46), (4, 46, 4, 23), (6, 24, 6, 32), (3, 13, 3, 100)])
def test_other_strides(lib, na, sa, nb, sb):
    V = 10
    for off in range(-nb * sb, na * sa):
        meets = any(i * sa < off + j * sb + V and off + j * sb < i * sa + V for i in range(na) for j in range(nb))
        rc = _probs(lib, AT, AT + off * 4, na, V, sa, sb)
        assert _taken(rc) if not meets else rc == cbq.CBQ_EINVAL, off


def test_between_the_rows(lib):
    """Ids in the columns behind the logits or the distributions."""
    n, V, st = 3, 10, 14
    for off in range(-4, 3 * st + 4):
        meets = any(i * st < off + n and off < i * st + V for i in range(n))
        far = AT + 0x10000
        for x, out in ((AT, far), (far, AT)):
            rc = _probs(lib, x, out, n, V, st, st, ids=AT + off * 4, u=far + 0x10000)
            assert _taken(rc) if not meets else rc == cbq.CBQ_EINVAL, off


def test_verify_rows(lib):
    """path, count and next in the columns behind p's and q's rows."""
    V, st, total, n, far = 10, 16, 4, 2, AT + 0x10000
    for off in range(-4, total * st + 4):
        meets = any(i * st < off + n and off < i * st + V for i in range(total))
        for p, q in ((AT, far), (far, AT)):
            rc = lib.cbq_verify(P(p), st, P(q), st, V, P(far + 0x1000), P(far + 0x2000), total, P(far + 0x3000), n, 3, P(far + 0x4000),
                                P(far + 0x5000), P(far + 0x6000), P(AT + off * 4), P(far + 0x7000), None, None)
            assert _taken(rc) if not meets else rc == cbq.CBQ_EINVAL, off
