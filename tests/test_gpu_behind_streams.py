"""The calls behind the logits on a stream of their own, inside a capture, and
two at a time, on the GPU; bits as on the current stream, one after another."""
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup
from tests.test_gpu_verify import _case
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu

HOLD = 20_000_000  # clocks: some 10 ms


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _i32(torch, *v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _calls(torch, seed=0):
    """Each: (call(stream) -> results, what it writes in place)."""
    calls = []
    for a in (([5000, 70], [40, 7], [5, 9], 32, 8, 128), ([6000, 300], [50, 0], [20, 9], 16, 2, 128), ([250], [9], [3], 8, 8, 128)):
        s = Setup(torch, *a, seed=seed)
        t = s.args()
        calls.append((lambda st, s=s, t=t: list(cbq.cbq_tree_attention8(*t, **s.limits, with_lse=True, stream=st)), []))
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, u = torch.randn((5, 50257), generator=g, device="cuda") * 3, torch.rand(5, generator=g, device="cuda")
    top = torch.full((5,), 0.9, device="cuda")
    calls.append((lambda st: list(cbq.cbq_probs(x, None, None, top, None, u=u, stream=st)), []))
    c = _case(torch, [5, 9, 1], 50257, 3 + seed)
    dev = [torch.from_numpy(c[k]).cuda() for k in ("tokens", "parent", "start", "u", "un")]
    calls.append((lambda st: list(cbq.cbq_verify(c["p"], c["q"], *dev, max_tok=9, stream=st)), []))
    kc, vc = (torch.randn((3, 9, 16, 2, 64), generator=g, device="cuda").bfloat16() for _ in "kv")
    table, path = torch.arange(9, dtype=torch.int32, device="cuda").flip(0).view(1, 9), _i32(torch, 0, 3, 5, 9, -1, -1, -1, -1, -1, -1)[None]
    calls.append((lambda st: [cbq.cbq_kv_commit(kc, vc, table, _i32(torch, 77), path, _i32(torch, 4), stream=st)], [kc, vc]))
    k16, v16 = (torch.randn((3, 9, 16, 2, 64), generator=g, device="cuda").bfloat16() for _ in "kv")
    k8, v8 = (torch.zeros((3, 9, 16, 2, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros((3, 9, 2, 2), device="cuda") for _ in "kv")
    src, dst = _i32(torch, 2, 0, 8), _i32(torch, 1, 8, 3)
    calls.append((lambda st: [cbq.cbq_kv_quantize(k16, v16, src, k8, v8, ks, vs, dst, stream=st) or ks], [k8, v8, ks, vs]))
    return calls


N = 7


def _same(torch, a, b):
    raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    return all(torch.equal(raw(x), raw(y)) for x, y in zip(a, b, strict=True))


def _fresh(torch, inplace, kept):
    for t, k in zip(inplace, kept):
        t.view(torch.uint8).copy_(k.view(torch.uint8))


def _once(torch, call, inplace, kept, stream=None):
    _fresh(torch, inplace, kept)
    torch.cuda.synchronize()
    got = call(stream)
    torch.cuda.synchronize()
    return [t.clone() for t in got + inplace]


@pytest.mark.parametrize("which", range(N))
def test_another_stream(torch, which):
    call, inplace = _calls(torch)[which]
    kept = [t.clone() for t in inplace]
    want = _once(torch, call, inplace, kept)
    sizes = sorted({t.numel() * t.element_size() for t in want} | {1 << 20, 8 << 20})
    side = torch.cuda.Stream()
    for _ in range(3):
        _fresh(torch, inplace, kept)
        torch.cuda.synchronize()
        # blocks that the current stream has freed and will write once more
        torch.cuda._sleep(HOLD)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD // 2)
        got = call(side)
        # the call's kernels wait; what it dropped must not be handed out here
        more = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert _same(torch, got + inplace, want)
        assert all(bool((t == 255).all()) for t in more)
        del got, more


@pytest.mark.parametrize("which", range(N))
def test_captured(torch, which):
    """Captured on a stream given by name and replayed; what is written in place is put back between."""
    call, inplace = _calls(torch)[which]
    kept = [t.clone() for t in inplace]
    want = _once(torch, call, inplace, kept)
    _fresh(torch, inplace, kept)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    if which == 5:  # (its small inputs are made inside the call: not inside a capture)
        ctx, count = _i32(torch, 77), _i32(torch, 4)
        kc, vc = inplace
        table, path = torch.arange(9, dtype=torch.int32, device="cuda").flip(0).view(1, 9), _i32(torch, 0, 3, 5, 9, -1, -1, -1, -1, -1, -1)[None]
        call = lambda st: [cbq.cbq_kv_commit(kc, vc, table, ctx, path, count, stream=st)]  # noqa: E731
        torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        got = call(side)
    for _ in range(3):
        _fresh(torch, inplace, kept)
        for t in got:
            if not any(t is x for x in inplace):
                t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert _same(torch, got + inplace, want)


@pytest.mark.parametrize("which", range(N))
def test_two_at_a_time(torch, which):
    """The call, and the same of other inputs, on two streams that nothing orders."""
    pairs = [_calls(torch, seed)[which] for seed in (0, 1)]
    kept = [[t.clone() for t in p[1]] for p in pairs]
    want = [_once(torch, p[0], p[1], k) for p, k in zip(pairs, kept)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for p, k in zip(pairs, kept):
            _fresh(torch, p[1], k)
        torch.cuda.synchronize()
        got = [p[0](s) for p, s in zip(pairs, sides)]
        torch.cuda.synchronize()
        for p, r, w in zip(pairs, got, want):
            assert _same(torch, r + p[1], w)
