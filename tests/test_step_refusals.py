"""The operators between the products refuse bad arguments before they touch
a GPU (CPU only), and the host table of a rotation holds its formulas."""
import ctypes
import math

import numpy as np
import pytest

from tests import step_ref
from verify_matvec_gb300 import build, cbq

P = ctypes.c_void_p
A = P(0x10000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cbq.load()


def _refused(fn, good, bad):
    """Each of `bad` (a dict of replaced arguments of the good call) gives EINVAL."""
    for change in bad:
        args = dict(good, **change)
        assert fn(*args.values()) == cbq.CBQ_EINVAL, change


def test_rope_refusals(lib):
    good = dict(x=A, dtype=0, n=4, heads=2, dim=8, xt=16, xh=8, pos=A, turns=A, rot=8, off=0, layout=0, m=1.0,
                out=P(0x20000), ot=16, oh=8, stream=None)
    _refused(lib.cbq_rope, good, [
        dict(x=None), dict(out=None), dict(pos=None), dict(turns=None), dict(dtype=3), dict(dtype=-1), dict(n=0),
        dict(n=(1 << 24) + 1), dict(heads=0), dict(heads=65536), dict(dim=0), dict(dim=1025), dict(xt=-1),
        dict(oh=-1), dict(rot=0), dict(rot=7), dict(rot=10), dict(off=-2), dict(off=2), dict(layout=2),
        dict(layout=-1), dict(m=math.inf), dict(m=math.nan), dict(x=P(0x10002)), dict(pos=P(0x10002)),
        dict(turns=P(0x10004)), dict(out=A, ot=32), dict(out=A, oh=4)])


def _cache(**change):
    c = dict(k=0x30000, v=0x40000, dtype=1, kv_heads=2, head_dim=8, page_size=4, n_pages=3, page_stride=64,
             tok_stride=16, head_stride=8)
    return ctypes.byref(cbq.cbq_kv_cache(*dict(c, **change).values()))


BAD_CACHES = [dict(k=None), dict(v=None), dict(dtype=0), dict(dtype=7), dict(kv_heads=0), dict(kv_heads=257),
              dict(head_dim=0), dict(head_dim=257), dict(page_size=0), dict(n_pages=0), dict(n_pages=1 << 31),
              dict(page_stride=-1), dict(tok_stride=-1), dict(head_stride=-1), dict(k=0x30001), dict(v=0x40001)]


def test_rope_append_refusals(lib):
    good = dict(q=A, k=A, v=A, dtype=0, n=4, heads=4, qt=32, qh=8, kt=16, kh=8, pos=A, slots=A, turns=A, rot=8, off=0,
                layout=0, m=1.0, cache=_cache(), out=P(0x20000), err=None, stream=None)
    _refused(lib.cbq_rope_append, good, [
        dict(q=None), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(turns=None), dict(out=None),
        dict(cache=None), dict(dtype=5), dict(n=0), dict(heads=0), dict(qt=-1), dict(kh=-1), dict(rot=3),
        dict(rot=10), dict(off=1), dict(layout=5), dict(m=math.nan), dict(slots=P(0x10004)), dict(k=P(0x10002)),
        dict(out=P(0x20001)), dict(err=P(0x10002))] + [dict(cache=_cache(**c)) for c in BAD_CACHES])


def test_tree_attention_refusals(lib):
    good = dict(q=A, qt=32, qh=8, heads=4, total=3, cache=_cache(), table=A, width=2, n_seq=1, ctx=A, start=A, mask=A,
                max_tok=3, max_len=8, scale=1.0, out=P(0x20000), out_dtype=1, lse=None, ws=A, ws_bytes=1 << 40,
                err=None, stream=None)
    limits = [dict(heads=0), dict(heads=3), dict(heads=1026), dict(total=0), dict(total=(1 << 24) + 1), dict(n_seq=0),
              dict(n_seq=65536), dict(max_tok=0), dict(max_tok=65), dict(max_len=0), dict(max_len=(1 << 30) + 1)]
    _refused(lib.cbq_tree_attention, good, limits + [
        dict(q=None), dict(table=None), dict(ctx=None), dict(start=None), dict(mask=None), dict(out=None),
        dict(ws=None), dict(cache=None), dict(qt=-1), dict(qh=-1), dict(width=0), dict(scale=math.inf),
        dict(out_dtype=2), dict(out_dtype=9), dict(ws=P(0x10008)), dict(ws_bytes=0), dict(mask=P(0x10004)),
        dict(q=P(0x10001)), dict(lse=P(0x10002)), dict(err=P(0x10002))] + [dict(cache=_cache(**c)) for c in BAD_CACHES])
    b = ctypes.c_int64()
    good = dict(n_seq=1, total=3, max_tok=3, max_len=8, heads=4, kv=2, dim=8, bytes=ctypes.byref(b))
    assert lib.cbq_tree_attention_workspace(*good.values()) == cbq.CBQ_OK and b.value >= 16
    _refused(lib.cbq_tree_attention_workspace, good, limits + [dict(kv=0), dict(kv=257), dict(dim=0), dict(dim=257),
                                                               dict(bytes=None)])


def test_sample_refusals(lib):
    good = dict(x=A, dtype=0, n=2, V=10, stride=10, t=None, k=None, p=None, m=None, u=A, ids=A, probs=None, stream=None)
    _refused(lib.cbq_sample, good, [
        dict(x=None), dict(u=None), dict(ids=None), dict(dtype=3), dict(n=0), dict(n=65536), dict(V=0),
        dict(V=cbq.CBQ_SAMPLE_MAX_V + 1, stride=1 << 20), dict(stride=9), dict(n=1, stride=-1), dict(x=P(0x10002)),
        dict(t=P(0x10002)), dict(k=P(0x10002)), dict(p=P(0x10002)), dict(m=P(0x10002)), dict(u=P(0x10002)),
        dict(ids=P(0x10002)), dict(probs=P(0x10002))])


def _turns(rot, **how):
    return cbq.cbq_rope_turns(rot, device="cpu", **how).numpy()


@pytest.mark.parametrize("rot", [2, 64, 128, 1024])
def test_turns(lib, rot):
    t, factor, length, low, high = step_ref.turns(rot, 500000.0), 8.0, 4096.0, 1.0, 4.0
    np.testing.assert_allclose(_turns(rot, base=500000.0), t, rtol=1e-13)
    np.testing.assert_allclose(_turns(rot, base=500000.0, scaling="linear", factor=factor), t / factor, rtol=1e-13)
    how = dict(base=500000.0, factor=factor, orig_len=length, low=low, high=high)
    got = _turns(rot, scaling="turns", **how)
    laps = t * length
    np.testing.assert_allclose(got[laps >= high], t[laps >= high], rtol=1e-13)
    np.testing.assert_allclose(got[laps <= low], t[laps <= low] / factor, rtol=1e-13)
    mid = (laps > low) & (laps < high)
    g = (laps[mid] - low) / (high - low)
    np.testing.assert_allclose(got[mid], g * t[mid] + (1 - g) * t[mid] / factor, rtol=1e-12)
    got = _turns(rot, scaling="index", **how)
    g = (got / t - 1 / factor) / (1 - 1 / factor)  # the part that stays
    assert np.all((g >= -1e-12) & (g <= 1 + 1e-12)) and np.all(np.diff(g) <= 1e-12)
    if rot >= 64:  # whole above `high` laps and gone one index past `low`
        assert np.all(g[laps > high * 1.5] > 0.99) and np.all(g[laps < low / 1.5] < 0.01)


def test_turns_refusals(lib):
    out = np.zeros(64)
    good = dict(rot=8, base=1e4, scaling=2, factor=4.0, length=4096.0, low=1.0, high=4.0, out=out.ctypes.data_as(P))
    assert lib.cbq_rope_turns(*good.values()) == cbq.CBQ_OK
    _refused(lib.cbq_rope_turns, good, [
        dict(rot=0), dict(rot=7), dict(rot=1026), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
        dict(scaling=-1), dict(scaling=4), dict(factor=0.0), dict(factor=math.nan), dict(length=0.0), dict(low=0.0),
        dict(low=4.0), dict(high=math.inf), dict(out=None)])
    with pytest.raises(ValueError):
        cbq.cbq_rope_turns(8, scaling="other", device="cpu")
