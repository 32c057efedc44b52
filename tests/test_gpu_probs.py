"""Distributions (cbq_probs) on the GPU against the definition in 64 bits.  A
weight is held within 2^-38 of itself and 2^-46 (of the largest, 1), the quotient
within 2^-23: with w of a kept mass m, |p - w/m| <= (2^-23 + 2^-37) w/m + 2^-46/m,
and m >= 1.  Rows in which a cut comes nearer than 2^-30 to falling elsewhere are
left out, and few may be."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _go(torch, logits, t=None, k=None, p=None, m=None, draw=True, most_near=1):
    n, V = logits.shape
    dev = lambda a, d: None if a is None else torch.tensor(a, dtype=d, device="cuda")  # noqa: E731
    how = dev(t, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(m, torch.float32)
    u = torch.from_numpy(np.random.default_rng(5).random(n, dtype=np.float32)).cuda()
    out, ids = Guarded(torch, (n, V), torch.float32), Guarded(torch, (n,), torch.int32)
    out.view.fill_(float("nan"))
    if draw:
        cbq.cbq_probs(logits, *how, u=u, out=out.view, ids=ids.view)
        assert torch.equal(ids.view, cbq.cbq_sample(logits, *how, u)[0])  # the same draw
    else:
        cbq.cbq_probs(logits, *how, out=out.view)
    torch.cuda.synchronize()
    out.check()
    ids.check()
    got, rows, near = out.view.double().cpu().numpy(), logits.double().cpu().numpy(), 0
    f = lambda a, i, d: d if a is None else float(np.float32(a[i]))  # noqa: E731
    for i in range(n):
        want, margin = behind_ref.probs(rows[i], f(t, i, 1.0), int(f(k, i, 0)), f(p, i, 1.0), f(m, i, 0.0))
        if margin < 2.0 ** -30:
            near += 1
            continue
        off = np.abs(got[i] - want) - (2.0 ** -23 + 2.0 ** -37) * want - 2.0 ** -46
        assert np.all(off <= 0), (i, int(np.argmax(off)), got[i][np.argmax(off)], want[np.argmax(off)])
        assert np.all(got[i][want == 0] <= 2.0 ** -46)
    assert near <= most_near
    return got


def _logits(torch, n, V, seed, dtype="float32", scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, V), generator=g, device="cuda") * scale).to(getattr(torch, dtype))


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 8193, 50257, 129280, 262144])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_sizes_and_types(torch, V, dtype):
    n = 9
    x = _logits(torch, n, V, V, dtype)
    _go(torch, x)
    _go(torch, x, t=[0.7] * n, draw=False)
    _go(torch, x, t=[0.8] * n, k=[1, 2, 5, 40, 1000, V, V + 5, 0, -3], most_near=0)
    if dtype == "float32":  # (16-bit logits have equal ones at every border)
        _go(torch, x, t=[0.9] * n, p=[0.0, 1e-6, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0, 2.0])
    _go(torch, x, m=[0.0, 1e-8, 1e-3, 0.05, 0.1, 0.5, 0.999, 1.0, 3.0], draw=False, most_near=2)
    _go(torch, x, t=[0.0, -1.0, float("nan"), 1.0, 1e-30, 1e30, float("inf"), 1e-3, 1e3])


@pytest.mark.parametrize("n", [1, 5, 24, 25, 150, 400])
def test_rows(torch, n):
    """From many blocks a row to one, all cuts."""
    rng = np.random.default_rng(n)
    x = _logits(torch, n, 5003, n)
    _go(torch, x, t=list(rng.uniform(0.3, 1.5, n)), k=[int(v) for v in rng.integers(0, 1200, n)],
        p=list(rng.uniform(0.3, 1.1, n)), m=list(rng.uniform(0, 0.05, n)), most_near=2)
    _go(torch, x, t=[1.3] * n, p=[0.9999] * n, most_near=2)


def test_what_has_no_place(torch):
    """Rows of -inf and NaN, of +inf among them, of one value, of ties at the cut."""
    inf, nan, V = float("inf"), float("nan"), 3001
    x = _logits(torch, 8, V, 1)
    x[0] = -inf
    x[1] = nan
    x[2, 7:] = -inf
    x[3, 100], x[3, 2000], x[3, 5] = inf, inf, nan
    x[4] = 1.5
    x[5] = (x[5] * 2).round()  # many equal ones
    x[6, 17] = nan
    for how in (dict(), dict(k=[5] * 8), dict(t=[0.0] * 8)):
        got = _go(torch, x, **how)
        assert not got[0].any() and not got[1].any()
        if how.get("t") is None:
            assert got[3][100] == got[3][2000] == 0.5
        if "k" in how:
            assert np.array_equal(np.flatnonzero(got[4]), np.arange(5)) and np.count_nonzero(got[5]) == 5
    got = _go(torch, x[4:5], p=[0.25])  # of V equal ones the first quarter
    assert np.array_equal(np.flatnonzero(got[0]), np.arange(-(-V // 4)))


def test_strides_and_places(torch):
    """Rows inside wider tensors, from an odd place on, on both sides."""
    for dtype in ("float32", "bfloat16"):
        x = _logits(torch, 6, 7001, 3, dtype)[:, 3:6004]
        want = cbq.cbq_probs(x.contiguous(), None, None, torch.full((6,), 0.9, device="cuda"), None)
        wide = torch.full((6, 6100), 7.0, device="cuda")
        got = cbq.cbq_probs(x, None, None, torch.full((6,), 0.9, device="cuda"), None, out=wide[:, 5:6006])
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool((wide[:, :5] == 7).all()) and bool((wide[:, 6006:] == 7).all())


def test_refusals(torch):
    x = _logits(torch, 4, 100, 1)
    u = torch.rand(4, device="cuda")
    with pytest.raises(ValueError):
        cbq.cbq_probs(x, None, None, None, None, ids=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        cbq.cbq_probs(x, None, None, None, None, out=torch.zeros((4, 99), device="cuda"))
    with pytest.raises(ValueError):
        cbq.cbq_probs(x.t().contiguous().t(), None, None, None, None)
    with pytest.raises(TypeError):
        cbq.cbq_probs(x.double(), None, None, None, None)
    with pytest.raises(TypeError):
        cbq.cbq_probs(x, u.double(), None, None, None)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_probs(x, None, None, None, None, out=x)
