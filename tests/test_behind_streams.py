"""Where the calls behind the logits take memory from when they are given a
stream that is not torch's current one (CPU only, as tests/test_step_streams.py)."""
import pytest
import torch

from tests.test_step_streams import Stream, _t, seen  # noqa: F401
from verify_matvec_gb300 import cbq

I32 = torch.int32


@pytest.fixture(autouse=True)
def real_sizes(seen, monkeypatch):  # noqa: F811
    """The size of a workspace is the library's own answer."""
    fake, real = cbq.load(), cbq._lib

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name) if name == "cbq_tree_attention8_workspace" else getattr(fake, name)

    monkeypatch.setattr(cbq, "load", Lib)
    cbq.cbq_tree_attention8_workspace.cache_clear()


def _cache8(pages, page, heads, dim):
    return ([_t(pages, page, heads, dim, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in "kv"],
            [_t(pages, 1, heads) for _ in "kv"])


def _probs(stream):
    return list(cbq.cbq_probs(_t(3, 50), None, None, None, None, u=_t(3), stream=stream))


def _verify(stream):
    return list(cbq.cbq_verify(_t(5, 50), _t(5, 50), _t(5, dtype=I32), _t(5, dtype=I32), _t(3, dtype=I32), _t(5), _t(2),
                               max_tok=4, stream=stream))


def _commit(stream):
    c = [_t(2, 3, 4, 1, 8, dtype=torch.bfloat16) for _ in "kv"]
    return [cbq.cbq_kv_commit(*c, _t(2, 3, dtype=I32), _t(2, dtype=I32), _t(2, 4, dtype=I32), _t(2, dtype=I32), stream=stream)]


def _quantize(stream):
    c8, s = _cache8(3, 4, 1, 8)
    cbq.cbq_kv_quantize(*[_t(3, 4, 1, 8, dtype=torch.bfloat16) for _ in "kv"], _t(2, dtype=I32), *c8, *s, _t(2, dtype=I32), stream=stream)
    return []


def _attention8(stream):
    c8, s = _cache8(128, 64, 1, 128)
    c = [_t(8, 64, 1, 128, dtype=torch.bfloat16) for _ in "kv"]
    return list(cbq.cbq_tree_attention8(_t(5, 4, 128, dtype=torch.bfloat16), *c8, *s, _t(1, 128, dtype=I32), _t(1, dtype=I32), *c,
                                        _t(1, 130, dtype=I32), _t(1, dtype=I32), _t(2, dtype=I32), _t(5, dtype=torch.int64),
                                        max_tok=5, max_old=8000, max_new=100, with_lse=True, stream=stream))


CALLS = dict(probs=_probs, verify=_verify, commit=_commit, quantize=_quantize, attention8=_attention8)


@pytest.mark.parametrize("call", CALLS)
def test_memory_is_the_streams_own(seen, call):  # noqa: F811
    s = Stream()
    returned = CALLS[call](s)
    assert seen["launched"] == [s.cuda_stream]
    assert all(under is s for _, under in seen["taken"]), "taken from another stream's pool"
    assert len(seen["taken"]) == len(returned) + (call == "attention8")  # (and a workspace: the keys are split)
    used = [t.data_ptr() for t, stream in seen["used"] if stream == "current"]
    assert all(t.data_ptr() in used for t in returned), "handed out without a word to the allocator"


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_needs_nothing(seen, call):  # noqa: F811
    CALLS[call](None)
    assert seen["launched"] == [0xC0]
    assert all(under is None for _, under in seen["taken"]) and not seen["used"]
