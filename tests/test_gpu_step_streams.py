"""The calls between the products on a stream of their own, on the GPU: while
that stream is held up, the current one takes memory of the sizes that the
call took and writes all over it, and memory that the current one has freed,
but not yet written for the last time, is no place for the call's results.
Bits as on the current stream."""
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention import Setup
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu

HOLD = 20_000_000  # clocks: some 10 ms


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _calls(torch):
    s = Setup(torch, [5000, 77], [5, 9], 32, 8, 128, 16)  # split over blocks and joined
    assert cbq.cbq_tree_attention_workspace(2, 14, 9, s.max_len, 32, 8, 128) > 1 << 20
    w = Setup(torch, [6000, 300], [20, 9], 16, 2, 128, 16)
    x = torch.randn((40, 8, 128), device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    slots = pos.long()
    turns = cbq.cbq_rope_turns(128)
    kv = [torch.zeros((8, 16, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    logits, u = torch.randn((5, 50257), device="cuda"), torch.rand(5, device="cuda")
    k = torch.full((5,), 40, dtype=torch.int32, device="cuda")
    sets = [(a, a.dev()) for a in (s, w)]
    calls = [lambda st, a=a, d=d: list(cbq.cbq_tree_attention(a.q, a.kc, a.vc, *d, max_tok=a.max_tok, max_len=a.max_len,
                                                              with_lse=True, stream=st)) for a, d in sets]
    calls.append(lambda st: [cbq.cbq_rope(x, pos, turns, stream=st)])
    calls.append(lambda st: [cbq.cbq_rope_append(x, x, x, pos, slots, turns, *kv, stream=st)])
    calls.append(lambda st: list(cbq.cbq_sample(logits, None, k, None, None, u, stream=st)))
    return calls


@pytest.mark.parametrize("which", range(5))
def test_another_stream(torch, which):
    call = _calls(torch)[which]
    want = [t.clone() for t in call(None)]
    sizes = sorted({t.numel() * t.element_size() for t in want} | {1 << 20, 8 << 20, 16 << 20})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks that the current stream has freed and will write once more
        torch.cuda._sleep(HOLD)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD // 2)
        got = call(side)
        # the call's kernels wait; what it dropped must not be handed out here
        kept = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((t == 255).all()) for t in kept)
        del got, kept


@pytest.mark.parametrize("which", range(5))
def test_results_go_back_when_the_current_stream_is_done(torch, which):
    """A result used on the current stream and dropped there: the next call on
    the other stream must not get its memory before that use is over."""
    call = _calls(torch)[which]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    copies = []
    for _ in range(4):
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(HOLD // 4)
        copies.append([t.clone() for t in got])  # (read late)
        del got
        with torch.cuda.stream(side):
            junk = [torch.full_like(t, 7) for t in want]
        del junk
    torch.cuda.synchronize()
    for c in copies:
        assert all(torch.equal(a, b) for a, b in zip(c, want))


def test_captured_on_another_stream(torch):
    """The calls inside a capture, on the capturing stream given by name."""
    for call in _calls(torch):
        want = [t.clone() for t in call(None)]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = call(side)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
