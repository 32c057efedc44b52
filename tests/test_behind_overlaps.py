"""Outputs of what follows a verify step's logits that overlap what the call
reads, or one another, are refused before a GPU is touched: blocks of other
rows or sequences would still read what one has written (CPU only)."""
import ctypes

import pytest

from tests.test_step_refusals import _cache
from verify_matvec_gb300 import build, cbq

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cbq.load()


def _places(*sizes):
    """Non-overlapping buffers, end to end, of the given bytes."""
    at, out = 0x100000, []
    for n in sizes:
        out.append(at)
        at += n
    return out


def _run(fn, args, sizes, outs):
    """Buffers side by side pass the check of overlaps (and get no further than
    the check for a GPU, or, on one, are not run here); an output moved onto
    another buffer's first or last word is refused."""
    names = list(sizes)
    where = dict(zip(names, _places(*sizes.values())))
    call = lambda w: fn(*[P(w[a]) if isinstance(a, str) and a in w else a for a in args])  # noqa: E731
    for o in outs:
        for n in names:
            if n == o:
                continue
            for at in (where[n], where[n] + sizes[n] - 4, where[n] - sizes[o] + 4):
                assert call(dict(where, **{o: at})) == cbq.CBQ_EINVAL, (o, n, at - where[n])
    return call(where)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_probs(lib):
    n, V, st = 3, 10, 12
    sizes = {"x": (2 * st + V) * 4, "t": 12, "k": 12, "p": 12, "m": 12, "u": 12, "out": (2 * st + V) * 4, "ids": 12}
    args = ["x", 0, n, V, st, "t", "k", "p", "m", "u", "out", st, "ids", None]
    if _no_gpu():
        assert _run(lib.cbq_probs, args, sizes, ["out", "ids"]) not in (cbq.CBQ_OK, cbq.CBQ_EINVAL)


def test_verify(lib):
    sizes = {"p": (3 * 12 + 10) * 4, "q": (3 * 16 + 10) * 4, "tokens": 16, "parent": 16, "start": 12, "u": 16,
             "un": 8, "path": 24, "count": 8, "next": 8}
    args = ["p", 12, "q", 16, 10, "tokens", "parent", 4, "start", 2, 3, "u", "un", "path", "count", "next", None, None]
    if _no_gpu():
        assert _run(lib.cbq_verify, args, sizes, ["path", "count", "next"]) not in (cbq.CBQ_OK, cbq.CBQ_EINVAL)


def test_commit(lib):
    sizes = {"table": 2 * 3 * 4, "ctx": 8, "path": 2 * 3 * 4, "count": 8, "out": 8}
    args = [_cache(), 2, 192, "table", 3, 2, "ctx", "path", 3, "count", "out", None, None]
    if _no_gpu():
        assert _run(lib.cbq_kv_commit, args, sizes, ["out"]) not in (cbq.CBQ_OK, cbq.CBQ_EINVAL)
