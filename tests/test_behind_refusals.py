"""What follows a verify step's logits refuses bad arguments before it touches a
GPU (CPU only), and the rule of the verification gives the target's distribution."""
import ctypes

import numpy as np
import pytest

from tests import behind_ref
from tests.test_step_refusals import BAD_CACHES, _cache, _refused
from verify_matvec_gb300 import build, cbq

P = ctypes.c_void_p
A = P(0x10000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cbq.load()


def test_probs_refusals(lib):
    good = dict(x=A, dtype=0, n=2, V=10, stride=10, t=None, k=None, p=None, m=None, u=None, out=P(0x20000), so=10,
                ids=None, stream=None)
    _refused(lib.cbq_probs, good, [
        dict(x=None), dict(out=None), dict(u=A), dict(ids=A), dict(dtype=3), dict(n=0), dict(n=65536), dict(V=0),
        dict(V=cbq.CBQ_SAMPLE_MAX_V + 1, stride=1 << 20, so=1 << 20), dict(stride=9), dict(so=9), dict(n=1, stride=-1),
        dict(n=1, so=-1), dict(x=P(0x10002)), dict(t=P(0x10002)), dict(k=P(0x10002)), dict(p=P(0x10002)),
        dict(m=P(0x10002)), dict(u=P(0x10002), ids=A), dict(u=A, ids=P(0x10002)), dict(out=P(0x20002)),
        dict(out=A), dict(out=P(0x10000 + 76)), dict(out=P(0x10000 - 76)), dict(dtype=1, out=P(0x10000 + 36))])


def test_verify_refusals(lib):
    good = dict(p=A, ps=10, q=A, qs=10, V=10, tokens=A, parent=A, total=4, start=A, n_seq=2, max_tok=3, u=A, un=A,
                path=A, count=A, next=A, err=None, stream=None)
    _refused(lib.cbq_verify, good, [
        dict(p=None), dict(tokens=None), dict(parent=None), dict(start=None), dict(u=None), dict(un=None),
        dict(path=None), dict(count=None), dict(next=None), dict(ps=9), dict(qs=9), dict(total=1, ps=-1),
        dict(total=1, qs=-1), dict(V=0), dict(V=cbq.CBQ_SAMPLE_MAX_V + 1, ps=1 << 20, qs=1 << 20), dict(total=0),
        dict(total=(1 << 24) + 1), dict(n_seq=0), dict(n_seq=65536), dict(max_tok=0), dict(max_tok=65)] + [
        {x: P(0x10002)} for x in ("p", "q", "tokens", "parent", "start", "u", "un", "path", "count", "next", "err")])


def test_commit_refusals(lib):
    good = dict(cache=_cache(), layers=2, ls=192, table=A, width=2, n_seq=1, ctx=A, path=A, max_tok=3, count=A,
                out=P(0x20000), err=None, stream=None)
    _refused(lib.cbq_kv_commit, good, [
        dict(cache=None), dict(layers=0), dict(layers=65536), dict(ls=-1), dict(table=None), dict(width=0),
        dict(n_seq=0), dict(n_seq=65536), dict(ctx=None), dict(path=None), dict(max_tok=0), dict(max_tok=65),
        dict(count=None), dict(out=A)] + [dict(cache=_cache(**c)) for c in BAD_CACHES] + [
        {x: P(0x10002)} for x in ("table", "ctx", "path", "count", "out", "err")])


def cache8(**change):
    c = dict(k=0x30001, v=0x40001, ks=0x50000, vs=0x60000, kv_heads=2, head_dim=8, page_size=4, block=2, n_pages=3,
             page_stride=64, tok_stride=16, head_stride=8, scale_page=4, scale_block=2, scale_head=1)
    return ctypes.byref(cbq.cbq_kv_cache8(*dict(c, **change).values()))


BAD_CACHES8 = [dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(ks=0x50002), dict(vs=0x50002),
               dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=0), dict(head_dim=257), dict(page_size=0),
               dict(block=0), dict(block=3), dict(block=8), dict(n_pages=0), dict(n_pages=1 << 30),
               dict(page_stride=-1), dict(tok_stride=-1), dict(head_stride=-1), dict(scale_page=-1),
               dict(scale_block=-1), dict(scale_head=-1), dict(page_size=1 << 17, block=1 << 17)]


def test_quantize_refusals(lib):
    good = dict(a=_cache(), ls=192, src=A, b=cache8(), ls8=192, lss=12, dst=A, layers=2, n=2, err=None, stream=None)
    _refused(lib.cbq_kv_quantize, good, [
        dict(a=None), dict(b=None), dict(ls=-1), dict(ls8=-1), dict(lss=-1), dict(src=None), dict(dst=None),
        dict(layers=0), dict(layers=65536), dict(n=0), dict(n=(1 << 24) + 1), dict(a=_cache(kv_heads=1)),
        dict(a=_cache(head_dim=4)), dict(a=_cache(page_size=8)), dict(src=P(0x10002)), dict(dst=P(0x10002)),
        dict(err=P(0x10002)), dict(n=1 << 24, a=_cache(kv_heads=256), b=cache8(kv_heads=256))] + [
        dict(a=_cache(**c)) for c in BAD_CACHES] + [dict(b=cache8(**c)) for c in BAD_CACHES8])


@pytest.mark.parametrize("k", [1, 2, 3, 7])
def test_what_comes_out_is_the_targets(k):
    """Drafts tried one after another, by the rule of the header, leave the
    target's distribution, whatever they were drawn from or chosen for."""
    rng = np.random.default_rng(k)
    for sharp in (0.3, 1.0, 4.0):
        p, q = (np.exp(sharp * rng.standard_normal(6)) for _ in "pq")
        p, q = p / p.sum(), q / q.sum()
        np.testing.assert_allclose(behind_ref.outcome(p, q, k), p, atol=1e-12)
        np.testing.assert_allclose(behind_ref.outcome(p, list(rng.integers(0, 6, k)), k), p, atol=1e-12)
        q[1] = 0.0
        np.testing.assert_allclose(behind_ref.outcome(p, q / q.sum(), k), p, atol=1e-12)


def test_the_references_rounding():
    """Of the reference itself: every e4m3 number is its own, halves go to even."""
    all_of = behind_ref._E4M3
    assert all_of[-1] == 448 and all_of[1] == 2.0 ** -9 and np.array_equal(behind_ref.e4m3(all_of), all_of)
    mid = (all_of[1:] + all_of[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, all_of[:-1], all_of[1:])
    assert np.array_equal(behind_ref.e4m3(mid), even) and np.array_equal(behind_ref.e4m3(-mid), -even)


def test_tree_attention8_refusals(lib):
    good = dict(q=A, qt=32, qh=8, heads=4, total=3, c8=cache8(), t8=A, w8=1, old=A, cache=_cache(), table=A, width=2,
                n_seq=1, ctx=A, start=A, mask=A, max_tok=3, max_old=4, max_new=8, scale=1.0, out=P(0x20000),
                out_dtype=1, lse=None, ws=A, ws_bytes=1 << 40, err=None, stream=None)
    limits = [dict(heads=0), dict(heads=3), dict(heads=1026), dict(total=0), dict(total=(1 << 24) + 1), dict(n_seq=0),
              dict(n_seq=65536), dict(max_tok=0), dict(max_tok=65), dict(max_old=-1), dict(max_old=(1 << 30) + 1),
              dict(max_old=1 << 30), dict(max_new=0), dict(max_new=(1 << 30) + 1), dict(max_new=(1 << 30) - 3)]
    _refused(lib.cbq_tree_attention8, good, limits + [
        dict(q=None), dict(t8=None), dict(old=None), dict(table=None), dict(ctx=None), dict(start=None),
        dict(mask=None), dict(out=None), dict(ws=None), dict(c8=None), dict(cache=None), dict(qt=-1), dict(qh=-1),
        dict(w8=0), dict(width=0), dict(scale=float("inf")), dict(out_dtype=2), dict(out_dtype=9), dict(ws=P(0x10008)),
        dict(ws_bytes=0), dict(mask=P(0x10004)), dict(q=P(0x10001)), dict(lse=P(0x10002)), dict(err=P(0x10002)),
        dict(t8=P(0x10002)), dict(old=P(0x10002)), dict(c8=cache8(kv_heads=1)), dict(c8=cache8(head_dim=4))] + [
        dict(cache=_cache(**c)) for c in BAD_CACHES] + [dict(c8=cache8(**c)) for c in BAD_CACHES8])
    b = ctypes.c_int64()
    good = dict(n_seq=1, total=3, max_tok=3, max_old=4, max_new=8, heads=4, kv=2, dim=8, bytes=ctypes.byref(b))
    assert lib.cbq_tree_attention8_workspace(*good.values()) == cbq.CBQ_OK and b.value >= 16
    _refused(lib.cbq_tree_attention8_workspace, good, limits + [dict(kv=0), dict(kv=257), dict(dim=0), dict(dim=257),
                                                                dict(bytes=None)])
    for old, new in ((1 << 29, 1 << 29), (0, 1 << 30), ((1 << 30) - 1, 1)):  # the ends: a plan is found at once
        for n_seq, heads in ((1, 2), (65535, 1024)):
            got = lib.cbq_tree_attention8_workspace(n_seq, 64, 64, old, new, heads, 2, 128, ctypes.byref(b))
            assert got == cbq.CBQ_OK and b.value >= 16
