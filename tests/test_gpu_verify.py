"""Verification (cbq_verify) on the GPU against the definition in 64 bits: the
same nodes and tokens, but where the definition comes nearer than 2^-40 of its
terms to another choice (sums are held within 2^-46 of theirs and V <= 2^18 terms
of random sign); such sequences are left out, and few may be."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _tree(rng, n, kind):
    """Parents of n nodes: a chain, a star (all behind node 0), or any tree."""
    if kind == "chain":
        return [-1] + list(range(n - 1))
    return [-1] + [0 if kind == "star" else int(rng.integers(0, i)) for i in range(1, n)]


def _case(torch, sizes, V, seed, kind="tree", drawn=True, sharp=2.0, near=0.7):
    """Device inputs of sequences of `sizes` nodes: the drafter's view is near the target's."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = max(1, sum(sizes))
    x = torch.randn((total, V), generator=g, device="cuda") * sharp
    p = torch.softmax(x, 1)
    q = torch.softmax(x + torch.randn((total, V), generator=g, device="cuda") * near, 1)
    start = np.cumsum([0] + list(sizes)).astype(np.int32)
    parent = np.array([v for n in sizes for v in _tree(rng, n, kind)[:n]] or [-1], np.int32)
    rows, tokens = q.double().cpu().numpy(), np.zeros(total, np.int32)
    for s, n in enumerate(sizes):
        for i in range(1, n):
            row = rows[start[s] + parent[start[s] + i]]
            tokens[start[s] + i] = rng.choice(V, p=row / row.sum())
    u, un = rng.random(total, dtype=np.float32), rng.random(max(1, len(sizes)), dtype=np.float32)
    return dict(p=p, q=q if drawn else None, tokens=tokens, parent=parent, start=start, u=u, un=un)


def _go(torch, c, max_tok, err=0, most_near=0):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    n = len(c["start"]) - 1
    path, count, nxt = (Guarded(torch, s, torch.int32) for s in ((n, max_tok), (n,), (n,)))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    cbq.cbq_verify(c["p"], c["q"], dev(c["tokens"]), dev(c["parent"]), dev(c["start"]), dev(c["u"]), dev(c["un"]),
                   max_tok=max_tok, path=path.view, count=count.view, next=nxt.view, err=word)
    torch.cuda.synchronize()
    for b in (path, count, nxt):
        b.check()
    assert int(word) == err
    p, q = (None if x is None else x.double().cpu().numpy() for x in (c["p"], c["q"]))
    got, counts, nexts, left_out = path.view.cpu().numpy(), count.view.cpu().numpy(), nxt.view.cpu().numpy(), 0
    for s in range(n):
        a, b = c["start"][s], c["start"][s + 1]
        if a < 0 or b < a or b > len(c["tokens"]) or a == b:
            assert counts[s] == 0 and nexts[s] == -1 and (got[s] == -1).all()
            continue
        b = min(b, a + max_tok)
        want, token, margin = behind_ref.verify(p[a:b], None if q is None else q[a:b], c["tokens"][a:b], c["parent"][a:b],
                                                c["u"][a:b], c["un"][s])
        if margin < 2.0 ** -40:
            left_out += 1
            continue
        assert counts[s] == len(want) and list(got[s][:len(want)]) == want and (got[s][len(want):] == -1).all(), (s, want, got[s])
        assert nexts[s] == token, (s, token, nexts[s], margin)
    assert left_out <= most_near
    return got, counts, nexts


@pytest.mark.parametrize("V", [1, 2, 5, 127, 129, 1000, 4099, 32000, 129280, 262144])
@pytest.mark.parametrize("drawn", [True, False])
def test_vocabularies(torch, V, drawn):
    for kind in ("chain", "star", "tree"):
        _go(torch, _case(torch, [5, 1, 9], V, V, kind, drawn), 9, most_near=1)


@pytest.mark.parametrize("sizes", [[1], [2], [64], [0, 3, 0], [64, 1, 33, 0, 7], [3] * 40, [2] * 200])
@pytest.mark.parametrize("drawn", [True, False])
def test_batches(torch, sizes, drawn):
    for kind in ("chain", "star", "tree"):
        for sharp, near in ((2.0, 0.7), (0.5, 0.2), (4.0, 3.0)):
            _go(torch, _case(torch, sizes, 517, len(sizes), kind, drawn, sharp, near), max(sizes), most_near=1)


@pytest.mark.parametrize("drawn", [True, False])
def test_every_child_is_accepted_or_refused(torch, drawn):
    """u = 0 takes each child that has any weight, u next to 1 hardly any; u_next at both ends."""
    for u in (0.0, 1.0 - 2.0 ** -24):
        for un in (0.0, 1.0 - 2.0 ** -24):
            for kind in ("chain", "star"):
                c = _case(torch, [9, 30], 1003, 3, kind, drawn, near=2.0)
                c["u"][:], c["un"][:] = u, un
                _, counts, _ = _go(torch, c, 30, most_near=2)
                if u == 0.0 and kind == "chain":
                    assert list(counts) == [9, 30]


def test_equal_tokens_among_the_children(torch):
    for drawn in (True, False):
        c = _case(torch, [12, 12], 50, 4, "star", drawn)
        c["tokens"][:] = 7
        c["u"][:] = 0.999
        _go(torch, c, 12)


def test_nothing_left(torch):
    """A target row under its drafter's everywhere (they do not sum to 1): drawn from the target; a row of zeros: -1."""
    c = _case(torch, [3, 3, 3], 8, 5, "star")
    c["p"][:] = 0
    c["q"][:] = 0.125
    c["p"][0, 2], c["p"][0, 5] = 0.0625, 0.0625
    c["p"][3:6, 1] = float("nan")
    c["p"][6, 4] = 1.0
    c["q"][6] = 0
    c["tokens"][:] = [0, 2, 5, 0, 1, 2, 0, 1, 3]
    c["u"][:] = 0.9
    c["un"][:] = [0.6, 0.5, 0.5]
    _, counts, nexts = _go(torch, c, 3)
    assert list(nexts) == [5, -1, 4] and list(counts) == [1, 1, 1]
    c["q"] = None
    c["tokens"][:] = [0, 2, 5, 0, 1, 2, 0, 4, 3]  # taken out: two, a NaN, all there is
    c["u"][:] = [0, 0.9, 0.9, 0, 0.9, 0.9, 0, 0.99, 0.9]
    c["p"][6, 4] = 0.5
    _go(torch, c, 3)


def test_tokens_and_parents_that_do_not_exist(torch):
    for drawn in (True, False):
        c = _case(torch, [6, 6], 40, 6, "star", drawn)
        c["tokens"][1], c["tokens"][2], c["tokens"][8] = -1, 40, 1 << 30
        c["parent"][3], c["parent"][4], c["parent"][9] = 3, 5, -7
        c["tokens"][0], c["parent"][0] = -9, 77  # node 0's are not looked at
        _go(torch, c, 6)


def test_lengths_that_do_not_fit(torch):
    bad = cbq.CBQ_DEVERR_BAD_LENGTH
    c = _case(torch, [4, 9, 2], 33, 7)
    _go(torch, c, 5, err=bad)  # one of 9 cut to 5
    c["start"][:] = [0, 4, 13, 16]  # the last leaves the rows
    _go(torch, c, 9, err=bad)
    c["start"][:] = [4, 0, 13, 15]  # one of less than no nodes
    _go(torch, c, 13, err=bad)
    c["start"][:] = [-1, 4, 13, 15]
    _go(torch, c, 9, err=bad)


def test_strides_and_places(torch):
    """Rows inside wider tensors, from places that are not on 16 bytes: the same answers."""
    c = _case(torch, [5, 8], 1000, 8)
    want = _go(torch, c, 8)
    for off, width in ((1, 1003), (4, 1012), (2, 1001 + 2)):
        wide = [torch.full((13, width), 9.0, device="cuda") for _ in "pq"]
        d = dict(c)
        for w, k in zip(wide, "pq"):
            w[:, off:off + 1000] = c[k]
            d[k] = w[:, off:off + 1000]
        assert all(np.array_equal(a, b) for a, b in zip(want, _go(torch, d, 8)))


def test_refusals(torch):
    c = _case(torch, [3], 20, 9)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    good = [c["p"], c["q"], dev(c["tokens"]), dev(c["parent"]), dev(c["start"]), dev(c["u"]), dev(c["un"])]
    cbq.cbq_verify(*good, max_tok=3)
    for i, x, e in ((0, c["p"].double(), TypeError), (1, c["q"].half(), TypeError), (0, c["p"].cpu(), TypeError),
                    (1, c["q"][:, :19], ValueError), (0, c["p"].t().contiguous().t(), ValueError),
                    (2, good[2].long(), TypeError), (3, good[3][:2], ValueError), (5, good[5][:2], ValueError),
                    (6, torch.rand(2, device="cuda"), ValueError)):
        args = list(good)
        args[i] = x
        with pytest.raises(e):
            cbq.cbq_verify(*args, max_tok=3)
    for n in (0, 65):
        with pytest.raises(cbq.CbqError):
            cbq.cbq_verify(*good, max_tok=n)
