"""Where the calls between the products take memory from when they are given a
stream that is not torch's current one (CPU only: the tensors stand in for
CUDA's, the launches do nothing).

The allocator hands a block that was freed to the next allocation of the same
stream without waiting for anybody's kernels.  So memory that a call takes for
kernels on `stream` has to come from that stream's pool, and what it returns,
which the caller goes on to use on the current stream, must be known to be in
use there."""
import contextlib

import pytest
import torch

from verify_matvec_gb300 import build, cbq


class OnGpu(torch.Tensor):
    is_cuda = True


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Stream:
    cuda_stream = 0x5EED


@pytest.fixture
def seen(monkeypatch):
    """What the calls allocate [(tensor, the stream it was taken under)], what they mark as in use [(tensor, stream)],
    and the streams that they launch on."""
    build.build()
    real, log = cbq.load(), {"taken": [], "used": [], "launched": [], "under": None}

    class Lib:
        def __getattr__(self, name):
            if name == "cbq_tree_attention_workspace":
                return getattr(real, name)

            def launch(*args):
                log["launched"].append(args[-1])
                return cbq.CBQ_OK
            return launch

    @contextlib.contextmanager
    def under(stream):
        was, log["under"] = log["under"], stream
        yield
        log["under"] = was

    empty = torch.empty

    def taking(*a, **k):
        t = empty(*a, **k).as_subclass(OnGpu)
        log["taken"].append((t, log["under"]))
        return t

    monkeypatch.setattr(cbq, "load", Lib)
    monkeypatch.setattr(torch, "empty", taking)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0xC0, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log["used"].append((t, s)))
    cbq._least_workspace.cache_clear()
    yield log
    cbq._least_workspace.cache_clear()


def _rope(stream):
    return [cbq.cbq_rope(_t(3, 2, 8), _t(3, dtype=torch.int32), _t(4, dtype=torch.float64), stream=stream)]


def _append(stream):
    c = [_t(2, 4, 1, 8, dtype=torch.bfloat16) for _ in "kv"]
    return [cbq.cbq_rope_append(_t(3, 2, 8), _t(3, 1, 8), _t(3, 1, 8), _t(3, dtype=torch.int32), _t(3, dtype=torch.int64),
                                _t(4, dtype=torch.float64), *c, stream=stream)]


def _attention(stream):
    c = [_t(128, 64, 1, 128, dtype=torch.bfloat16) for _ in "kv"]
    i32 = torch.int32
    return list(cbq.cbq_tree_attention(_t(5, 4, 128, dtype=torch.bfloat16), *c, _t(1, 128, dtype=i32), _t(1, dtype=i32),
                                       _t(2, dtype=i32), _t(5, dtype=torch.int64), max_tok=5, max_len=8000, with_lse=True,
                                       stream=stream))


def _sample(stream):
    return list(cbq.cbq_sample(_t(3, 50), None, None, None, None, _t(3), stream=stream))


CALLS = dict(rope=_rope, append=_append, attention=_attention, sample=_sample)


@pytest.mark.parametrize("call", CALLS)
def test_memory_is_the_streams_own(seen, call):
    s = Stream()
    returned = CALLS[call](s)
    assert seen["launched"] == [s.cuda_stream]
    assert seen["taken"] and all(under is s for _, under in seen["taken"]), "taken from another stream's pool"
    assert len(seen["taken"]) == len(returned) + (call == "attention")  # (and a workspace: the keys are split)
    used = [t.data_ptr() for t, stream in seen["used"] if stream == "current"]
    assert all(t.data_ptr() in used for t in returned), "handed out without a word to the allocator"


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_needs_nothing(seen, call):
    CALLS[call](None)
    assert seen["launched"] == [0xC0]
    assert all(under is None for _, under in seen["taken"]) and not seen["used"]
