"""Sampling (cbq_sample) on the GPU against the definition in 64 bits: the
same tokens, but where the definition itself comes nearer to another choice
than 2^-30 of the kept mass (its weights are held within 2^-39, and a row sums
up to 2^18 of them; such rows are left out, and few may be).  Probabilities
within 2^-23 of themselves (the last rounding, and the weights' 2^-39)."""
import numpy as np
import pytest

from tests import step_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _go(torch, logits, t=None, k=None, p=None, m=None, u=None, most_near=1):
    """logits: a CUDA tensor (n, V) of any type; the settings: lists, or None."""
    n = logits.shape[0]
    u = np.random.default_rng(7).random(n, dtype=np.float32) if u is None else np.asarray(u, dtype=np.float32)
    dev = lambda a, d: None if a is None else torch.tensor(a, dtype=d, device="cuda")  # noqa: E731
    gi, gp = Guarded(torch, (n,), torch.int32), Guarded(torch, (n,), torch.float32)
    cbq.cbq_sample(logits, dev(t, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(m, torch.float32),
                   torch.from_numpy(u).cuda(), ids=gi.view, probs=gp.view)
    torch.cuda.synchronize()
    gi.check()
    gp.check()
    ids, probs = gi.view.cpu().numpy(), gp.view.cpu().numpy()
    rows, near = logits.double().cpu().numpy(), 0
    f = lambda a, i, d: d if a is None else float(np.float32(a[i]))  # noqa: E731
    for i in range(n):
        want, prob, margin = step_ref.sample(rows[i], f(t, i, 1.0), int(f(k, i, 0)), f(p, i, 1.0), f(m, i, 0.0), float(u[i]))
        if margin < 2.0 ** -30:
            near += 1
            continue
        assert ids[i] == want, (i, ids[i], want, margin)
        assert abs(probs[i] - prob) <= 2.0 ** -23 * prob, (i, probs[i], prob)
    assert near <= most_near
    return ids, probs


def _logits(torch, n, V, seed, dtype="float32", scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, V), generator=g, device="cuda") * scale).to(getattr(torch, dtype))


SIZES = [1, 2, 3, 31, 33, 1000, 1025, 4097, 50257, 129280, 262144]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_sizes_and_types(torch, V, dtype):
    n = 9
    x = _logits(torch, n, V, V, dtype)
    _go(torch, x)
    _go(torch, x, t=[0.7] * n)
    _go(torch, x, t=[0.8] * n, k=[1, 2, 5, 40, 1000, V, V + 5, 0, -3])
    _go(torch, x, t=[0.9] * n, p=[0.0, 1e-6, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0, 2.0])
    _go(torch, x, m=[0.0, 1e-8, 1e-3, 0.05, 0.1, 0.5, 0.999, 1.0, 3.0])
    _go(torch, x, t=[0.5, 0.7, 0.9, 1.0, 1.1, 1.5, 2.0, 5.0, 0.05], k=[50, 0, 7, 200, 1, 3000, 64, 12, 90],
        p=[0.9, 0.5, 0.99, 0.3, 0.9, 0.95, 0.8, 0.7, 1.0], m=[0.01, 0.0, 0.1, 0.001, 0.2, 0.0, 0.05, 0.3, 0.02])
    _go(torch, x, t=[0.0, -1.0, float("nan"), 1.0, 1e-30, 1e30, float("inf"), 1e-3, 1e3])


@pytest.mark.parametrize("n", [1, 5, 64, 300])
def test_rows(torch, n):
    rng = np.random.default_rng(n)
    x = _logits(torch, n, 5003, n)
    _go(torch, x, t=list(rng.uniform(0.3, 1.5, n)), k=[int(v) for v in rng.integers(0, 400, n)],
        p=list(rng.uniform(0.3, 1.1, n)), m=list(rng.uniform(0, 0.05, n)))


def test_row_stride_and_offset(torch):
    """Rows inside a wider tensor, from an odd place on."""
    for dtype in ("float32", "bfloat16"):
        x = _logits(torch, 6, 7001, 3, dtype)
        _go(torch, x[:, 5:6006], t=[0.8] * 6, k=[30] * 6, p=[0.9] * 6)
        _go(torch, x[1:4, :999], t=[0.8] * 3, p=[0.9] * 3)


@pytest.mark.parametrize("V", [7, 5000, 129280])
def test_equal_logits(torch, V):
    """Ties go to the lowest index: top-k keeps the first k, top-p the first
    ceil(p V) of them, and u picks evenly among what is kept."""
    x = torch.full((6, V), -1.25, device="cuda")
    u = [0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.1]
    ids, _ = _go(torch, x, k=[4] * 6, u=u)
    np.testing.assert_array_equal(ids, [0, 1, 2, 3, 3, 0])
    _go(torch, x, p=[0.5, 0.25, 0.125, 0.75, 1e-9, 0.0], u=u)
    _go(torch, x, k=[5] * 6, p=[0.5] * 6, m=[1.0] * 6, u=u)
    ids, _ = _go(torch, x, m=[1.5] * 6, u=u)
    assert not ids.any()
    x[:, 3] = 2.0
    x[:, 5:] = -0.0
    x[:, 0] = 0.0
    _go(torch, x, k=[3] * 6, u=u)
    _go(torch, x, p=[0.9] * 6, u=u)


def test_few_values_many_ties(torch):
    """Logits on a coarse grid: every border falls inside ties."""
    for V in (100, 3001, 60000):
        x = torch.round(_logits(torch, 12, V, V) * 2) / 2
        rng = np.random.default_rng(V)
        _go(torch, x, t=[1.0] * 12, k=[int(v) for v in rng.integers(1, V, 12)])
        _go(torch, x, t=[0.7] * 12, p=list(rng.uniform(0.1, 0.99, 12)))
        _go(torch, x, t=[1.3] * 12, k=[int(v) for v in rng.integers(1, V, 12)], p=list(rng.uniform(0.1, 0.99, 12)))


def test_masked_and_odd_logits(torch):
    inf, nan = float("inf"), float("nan")
    x = _logits(torch, 8, 3000, 5)
    x[0, :] = -inf
    x[1, :] = nan
    x[2, :] = -inf
    x[2, 1234] = -3e38
    x[3, ::2] = -inf
    x[4, 7::3] = nan
    x[5, [10, 2000]] = inf
    x[6, :] = torch.finfo(torch.float32).min
    x[6, 77] = -1e38
    x[7, :] = torch.finfo(torch.float32).min
    for how in (dict(), dict(k=[3] * 8), dict(p=[0.7] * 8), dict(k=[2000] * 8, p=[0.9] * 8, m=[0.1] * 8), dict(t=[0.0] * 8)):
        ids, probs = _go(torch, x, **how)
        assert ids[0] == ids[1] == -1 and probs[0] == probs[1] == 0
        assert ids[2] == 1234


def test_every_token_at_its_share(torch):
    """u on a fine grid: each kept token is drawn in index order, as often as its probability says."""
    x = torch.tensor([[0.3, 2.0, -1.0, 2.0, 1.0, -5.0, 0.0]], device="cuda").repeat(4096, 1)
    u = (np.arange(4096) + 0.5) / 4096
    ids, probs = _go(torch, x, t=[0.8] * 4096, k=[5] * 4096, p=[0.95] * 4096, u=u)
    assert np.all(np.diff(ids) >= 0)
    for i in np.unique(ids):
        assert abs(np.mean(ids == i) - probs[ids == i][0]) <= 1 / 4096


def test_uniform_numbers_at_their_ends(torch):
    x = _logits(torch, 5, 2000, 6)
    _go(torch, x, u=[0.0, 2.0 ** -126, 1 - 2.0 ** -24, 2.0 ** -32, 0.5])
    ids, _ = _go(torch, x, k=[1] * 5, u=[0.0, 0.3, 1 - 2.0 ** -24, 0.7, 0.9])
    np.testing.assert_array_equal(ids, x.argmax(1).cpu().numpy())
    # outside [0, 1): as its nearest end
    d = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    a, _ = cbq.cbq_sample(x, None, None, None, None, d([-1.0, 1.0, 2.0, float("nan"), float("inf")]))
    assert torch.all((a >= 0) & (a < 2000))


def test_repeat_stream_graph_and_refusals(torch):
    x = _logits(torch, 5, 129280, 8)
    u = torch.rand(5, device="cuda")
    t, p = torch.full((5,), 0.9, device="cuda"), torch.full((5,), 0.9, device="cuda")
    k = torch.full((5,), 300, dtype=torch.int32, device="cuda")
    ids, probs = cbq.cbq_sample(x, t, k, p, None, u)
    for _ in range(3):
        a, b = cbq.cbq_sample(x, t, k, p, None, u)
        assert torch.equal(a, ids) and torch.equal(b, probs)
    into = torch.zeros_like(ids), torch.zeros_like(probs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cbq.cbq_sample(x, t, k, p, None, u, ids=into[0], probs=into[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(into[0], ids) and torch.equal(into[1], probs)
    with pytest.raises(ValueError):
        cbq.cbq_sample(x.T, t, k, p, None, u)
    with pytest.raises(ValueError):
        cbq.cbq_sample(x, t, k, p, None, u[:3])
    with pytest.raises(TypeError):
        cbq.cbq_sample(x, t, k.long(), p, None, u)
    with pytest.raises(TypeError):
        cbq.cbq_sample(x.double(), t, k, p, None, u)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_sample(torch.zeros((1, cbq.CBQ_SAMPLE_MAX_V + 1), device="cuda"), None, None, None, None, u[:1])


@pytest.mark.parametrize("V,dtype", [(1, "float32"), (33, "bfloat16"), (1001, "float32"), (4097, "float16"), (50257, "float32"), (129280, "bfloat16"),
                                     (262144, "float32")])
def test_many_rows(torch, V, dtype):
    """Enough rows that each is a block's own: every kind of setting, short and long rows, kept sets from one to all."""
    n = 60
    rng = np.random.default_rng(V)
    x = _logits(torch, n, V, V + 1, dtype)
    kinds = np.arange(n) % 6
    _go(torch, x, t=[0.0 if k == 5 else float(v) for k, v in zip(kinds, rng.uniform(0.3, 2.0, n))],
        k=[int(v) if k in (1, 4) else 0 for k, v in zip(kinds, np.exp(rng.uniform(0, np.log(V + 1), n)))],
        p=[float(v) if k in (2, 4) else 1.0 for k, v in zip(kinds, rng.uniform(0.05, 0.9999, n))],
        m=[float(v) if k in (3, 4) else 0.0 for k, v in zip(kinds, np.exp(rng.uniform(-12, 0.5, n)))])


def test_many_rows_strange(torch):
    """Ties, masks, odd strides and the odd values, a block a row."""
    inf, nan = float("inf"), float("nan")
    n, V = 64, 60001
    rng = np.random.default_rng(4)
    wide = torch.round(_logits(torch, n, V + 7, 9) * 2) / 2
    x = wide[:, 3:V + 3]
    x[0], x[1], x[2] = -inf, nan, 1.5
    x[3, ::2], x[4, 5::3], x[5, [7, 9000]] = -inf, nan, inf
    x[6] = -0.0
    x[6, 11::2] = 0.0
    x[7] = torch.finfo(torch.float32).min
    for how in (dict(), dict(k=[int(v) for v in rng.integers(1, V, n)]), dict(p=list(rng.uniform(0.01, 0.999, n))),
                dict(k=[int(v) for v in rng.integers(1, 50, n)], p=list(rng.uniform(0.1, 0.99, n)), m=list(rng.uniform(0, 0.3, n))),
                dict(t=[1e-3] * n, k=[40] * n), dict(t=[1e30] * n, p=[0.5] * n), dict(t=[inf] * n), dict(t=[0.0] * n)):
        ids, probs = _go(torch, x, **how)
        assert ids[0] == ids[1] == -1 and probs[0] == 0
    again = _go(torch, x, k=[100] * n, p=[0.9] * n)
    once = _go(torch, x, k=[100] * n, p=[0.9] * n)
    assert np.array_equal(again[0], once[0]) and np.array_equal(again[1], once[1])


def test_many_rows_dense_and_thin_stretches(torch):
    """What is kept fills some stretches of a row and leaves few or none in others."""
    n, V = 40, 70001
    rng = np.random.default_rng(11)
    x = _logits(torch, n, V, 17, scale=0.3)
    x[:, 1500:9000] += 6
    x[:, 40000:40300] += 6
    x[::2, 60000:60001] += 5
    for how in (dict(p=list(rng.uniform(0.3, 0.97, n))), dict(k=[int(v) for v in rng.integers(1, 9000, n)]), dict(m=[0.2] * n),
                dict(k=[7000] * n, p=list(rng.uniform(0.3, 0.99, n)), m=[0.02] * n)):
        _go(torch, x, u=rng.random(n, dtype=np.float32), **how)


@pytest.mark.parametrize("n", [3, 40])
def test_top_k_of_clustered_logits(torch, n):
    """The largest logits next to one another, a thread's own or a block's own; fewer of any weight than top-k takes."""
    V = 129280
    rng = np.random.default_rng(12)
    x = _logits(torch, n, V, 18, scale=0.5)
    x[:, 32 * 7::32][:, :200] += 9      # one lane's
    x[::3, 70000:70600] += 9.5          # one block's
    x[1] = -float("inf")
    x[1, 5:45] = torch.arange(40, device="cuda") / 8
    x[2, 100:130] = float("inf")
    for k in (1, 29, 30, 31, 39, 40, 41, 199, 511, 512, 513, 700):
        _go(torch, x, k=[k] * n, u=rng.random(n, dtype=np.float32))
    _go(torch, x, k=[int(v) for v in rng.integers(1, 800, n)], p=list(rng.uniform(0.3, 0.99, n)), u=rng.random(n, dtype=np.float32))
