"""Rotary positions and the append to a paged cache (cbq_rope,
cbq_rope_append) on the GPU against the definition in 64 bits.

Tolerance of a rotated value, in units of 2^-24 (|a| + |b|) |mscale|: the
part of a turn rounded to fp32 is off by 2^-26 turns, an angle of 1.6 units;
sine and cosine are within one ulp, 1 unit; their product with mscale, the
product with the value and the sum round, 0.5 units each: below 4.5, taken as
8.  One rounding to the output type (half a step, and the subnormal step of
fp16) comes on top."""
import numpy as np
import pytest

from tests import step_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _half_step(torch, dtype, want):
    if dtype == torch.float32:
        return 0.0
    return np.abs(want) * torch.finfo(dtype).eps / 2 + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def _check(torch, got, want, size, dtype, what="x"):
    got = got.double().cpu().numpy()
    lim = 8 * 2.0 ** -24 * size
    lim = lim + _half_step(torch, dtype, np.abs(want) + lim)
    bad = np.abs(got - want) > lim
    assert not bad.any(), f"{what}: {bad.sum()} off, first at {np.argwhere(bad)[0]}"


def _randn(torch, seed, *shape, dtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype or torch.float32)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("n,heads,dim,rot,off", [(1, 1, 2, 2, 0), (5, 32, 128, 128, 0), (3, 5, 192, 64, 128),
                                                 (7, 3, 80, 20, 30), (2, 1, 1024, 1024, 0), (130, 6, 96, 32, 64),
                                                 (9, 4, 67, 6, 1), (3, 70, 256, 64, 32), (2, 2, 72, 36, 12)])
def test_rope(torch, dtype, layout, n, heads, dim, rot, off):
    dt = getattr(torch, dtype)
    x = _randn(torch, n + dim, n, heads, dim, dtype=dt)
    pos = torch.randint(0, 1 << 17, (n,), dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(rot)
    g = Guarded(torch, x.shape, dt)
    cbq.cbq_rope(x, pos, t, rot_off=off, layout=layout, mscale=1.25, out=g.view)
    torch.cuda.synchronize()
    g.check()
    want, size = step_ref.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), off, layout, 1.25)
    _check(torch, g.view, want, size, dt)
    keep = np.r_[0:off, off + rot:dim]
    np.testing.assert_array_equal(g.view.double().cpu().numpy()[..., keep], x.double().cpu().numpy()[..., keep])


@pytest.mark.parametrize("pos", [[0, 1, -1, -70000], [2 ** 31 - 1, -2 ** 31, 1 << 20, 12345679]])
def test_far_positions(torch, pos):
    x = _randn(torch, 1, 4, 2, 64)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(64, scaling="turns", factor=16.0, orig_len=8192.0)
    want, size = step_ref.rotate(x.double().cpu().numpy(), np.array(pos), t.cpu().numpy(), 0, "half")
    _check(torch, cbq.cbq_rope(x, p, t), want, size, torch.float32)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_strides_alignment_and_in_place(torch, dtype, layout):
    """Heads that are a slice of a wider row, rows that start one value past an
    aligned place, heads-first memory, and the result in the input's place."""
    dt = getattr(torch, dtype)
    pos = torch.arange(50, 56, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(64)
    for base in (_randn(torch, 2, 6, 7, 200, dtype=dt)[:, 1:4, 3:131], _randn(torch, 3, 6, 3, 136, dtype=dt)[..., :128],
                 _randn(torch, 4, 3, 6, 128, dtype=dt).transpose(0, 1),
                 _randn(torch, 5, 6 * 3 * 128 + 1, dtype=dt)[1:].view(6, 3, 128)):
        want, size = step_ref.rotate(base.double().cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), 64, layout)
        got = cbq.cbq_rope(base, pos, t, rot_off=64, layout=layout)
        _check(torch, got, want, size, dt)
        assert cbq.cbq_rope(base, pos, t, rot_off=64, layout=layout, out=base) is base
        assert torch.equal(base, got)


@pytest.mark.parametrize("dtype,cache", [("float32", "bfloat16"), ("float32", "float16"), ("bfloat16", "bfloat16"),
                                         ("float16", "float16"), ("bfloat16", "float16"), ("float16", "bfloat16")])
@pytest.mark.parametrize("n,heads,kv,dim,rot,off,page", [(1, 1, 1, 8, 8, 0, 1), (5, 32, 8, 128, 128, 0, 64),
                                                         (33, 6, 3, 96, 32, 64, 7), (200, 10, 5, 67, 6, 1, 16)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append(torch, dtype, cache, n, heads, kv, dim, rot, off, page, heads_first):
    dt, cdt = getattr(torch, dtype), getattr(torch, cache)
    q, k, v = (_randn(torch, i + n, n, h, dim, dtype=dt) for i, h in enumerate((heads, kv, kv)))
    pages = 2 * n // page + 3
    shape = (pages, kv, page, dim) if heads_first else (pages, page, kv, dim)
    kc, vc = (_randn(torch, 9 + i, *shape, dtype=cdt) for i in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.randperm(pages * page, device="cuda")[:n]
    pos = torch.arange(1000, 1000 + n, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(rot)
    tt, pp, ss = t.cpu().numpy(), pos.cpu().numpy(), slots.cpu().numpy()
    kw, vw = kc.double().cpu().numpy().copy(), vc.double().cpu().numpy().copy()
    ks, vs = np.zeros_like(kw), np.zeros_like(vw)
    out = cbq.cbq_rope_append(q, k, v, pos, slots, t, kc, vc, rot_off=off, layout="pairs")
    want, size = step_ref.rotate(q.double().cpu().numpy(), pp, tt, off, "pairs")
    assert out.dtype == cdt
    _check(torch, out, want, size, cdt, "q")
    kw[ss // page, ss % page], ks[ss // page, ss % page] = step_ref.rotate(k.double().cpu().numpy(), pp, tt, off, "pairs")
    vw[ss // page, ss % page] = v.double().cpu().numpy()
    _check(torch, kc, kw, ks, cdt, "k")
    _check(torch, vc, vw, vs, cdt, "v")


def test_append_slots_that_are_none(torch):
    """A negative slot writes nothing; one beyond the cache writes nothing and is reported."""
    q, k, v = (_randn(torch, i, 4, 2, 16) for i in range(3))
    kc, vc = (_randn(torch, 5 + i, 3, 4, 2, 16, dtype=torch.bfloat16) for i in range(2))
    before = kc.clone(), vc.clone()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cbq.cbq_rope_append(q, k, v, pos, torch.tensor([-1, -2 ** 62, -5, 7], device="cuda"), t, kc, vc, err=err)
    assert err.item() == 0
    want, size = step_ref.rotate(q.double().cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), 0, "half")
    _check(torch, out, want, size, torch.bfloat16)
    same = torch.ones(12, dtype=torch.bool, device="cuda")
    same[7] = False
    for c, b in zip((kc, vc), before):
        assert torch.equal(c.flatten(0, 1)[same], b.flatten(0, 1)[same])
        assert not torch.equal(c.flatten(0, 1)[7], b.flatten(0, 1)[7])
    before = kc.clone(), vc.clone()
    cbq.cbq_rope_append(q, k, v, pos, torch.tensor([12, 2 ** 62, -1, 2 ** 32], device="cuda"), t, kc, vc, err=err)
    assert err.item() == cbq.CBQ_DEVERR_BAD_SLOT
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_nan_and_infinity_stay_in_their_pair(torch):
    x = _randn(torch, 8, 2, 2, 32)
    x[0, 0, 3], x[1, 1, 20] = float("nan"), float("inf")
    pos = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    y = cbq.cbq_rope(x, pos, cbq.cbq_rope_turns(32))
    odd = (~torch.isfinite(y)).nonzero().tolist()
    assert odd == [[0, 0, 3], [0, 0, 19], [1, 1, 4], [1, 1, 20]]


def test_stream_graph_and_refusals(torch):
    """On a stream of its own and replayed from a graph; what the binding refuses."""
    x = _randn(torch, 11, 40, 8, 128, dtype=torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(128)
    want = cbq.cbq_rope(x, pos, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cbq.cbq_rope(x, pos, t, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError):
        cbq.cbq_rope(x.transpose(1, 2), pos, t)
    with pytest.raises(ValueError):
        cbq.cbq_rope(x, pos[:3], t)
    with pytest.raises(TypeError):
        cbq.cbq_rope(x.double(), pos, t)
    with pytest.raises(TypeError):
        cbq.cbq_rope(x, pos.long(), t)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_rope(x, pos, t, rot_off=2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("n,heads,dim,rot,off", [(4801, 3, 64, 64, 0), (5000, 2, 96, 32, 64), (1700, 40, 128, 64, 64), (420, 9, 1024, 1024, 0)])
def test_many_tokens(torch, dtype, layout, n, heads, dim, rot, off):
    """Blocks that go through several tokens: an odd number of them, several parts of a token, heads turned in part."""
    test_rope(torch, dtype, layout, n, heads, dim, rot, off)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_many_tokens_strides_and_in_place(torch, layout):
    n = 4003
    pos = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)
    t = cbq.cbq_rope_turns(64)
    for base in (_randn(torch, 2, n, 5, 136, dtype=torch.bfloat16)[:, 1:4, :128], _randn(torch, 4, 3, n, 128).transpose(0, 1)):
        want, size = step_ref.rotate(base.double().cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), 64, layout)
        got = cbq.cbq_rope(base, pos, t, rot_off=64, layout=layout)
        _check(torch, got, want, size, base.dtype)
        assert cbq.cbq_rope(base, pos, t, rot_off=64, layout=layout, out=base) is base
        assert torch.equal(base, got)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_append_many_tokens(torch, dtype):
    """A prompt into a cache, with tokens that have no place in it."""
    test_append(torch, dtype, "float16", 4100, 4, 2, 64, 64, 0, 16, True)
    n, dt = 4100, getattr(torch, dtype)
    q, k, v = (_randn(torch, i, n, h, 64, dtype=dt) for i, h in enumerate((3, 1, 1)))
    kc, vc = (_randn(torch, 5 + i, 300, 16, 1, 64, dtype=torch.bfloat16) for i in range(2))
    before = kc.clone(), vc.clone()
    slots = torch.randperm(4800, device="cuda")[:n]
    slots[::3] = -1
    slots[4099] = 4800
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    t = cbq.cbq_rope_turns(32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cbq.cbq_rope_append(q, k, v, pos, slots, t, kc, vc, err=err)
    assert err.item() == cbq.CBQ_DEVERR_BAD_SLOT
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[::3] = False
    good[4099] = False
    for c, b, x in ((kc, before[0], cbq.cbq_rope(k, pos, t)), (vc, before[1], v)):
        b = b.view(4800, 1, 64)
        b[slots[good]] = x[good].to(torch.bfloat16) if x is v else b[slots[good]]
        if x is v:
            assert torch.equal(c.view(4800, 1, 64), b)
        else:
            rest = torch.ones(4800, dtype=torch.bool, device="cuda")
            rest[slots[good]] = False
            assert torch.equal(c.view(4800, 1, 64)[rest], b[rest])
            want, size = step_ref.rotate(k.double().cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), 0, "half")
            _check(torch, c.view(4800, 1, 64)[slots[good]], want[good.cpu().numpy()], size[good.cpu().numpy()], torch.bfloat16)
