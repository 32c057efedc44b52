"""The cache between two verify steps, on the GPU: the accepted drafts' move
(cbq_kv_commit) and pages turned into 8 bits (cbq_kv_quantize), both to the bit."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu
BAD_SLOT, BAD_LENGTH = cbq.CBQ_DEVERR_BAD_SLOT, cbq.CBQ_DEVERR_BAD_LENGTH


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _cache(torch, shape, seed, dtype="bfloat16", pad=0):
    """Random 16-bit values of any bits in a cache of that shape, its last axis inside one of dim + pad."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-(1 << 15), 1 << 15, (*shape[:-1], shape[-1] + pad), generator=g, device="cuda", dtype=torch.int16)
    return x.view(getattr(torch, dtype))[..., :shape[-1]]


def _bits(torch, x):
    return x.contiguous().view(torch.int16).cpu().numpy()


def _path(rng, n, most):
    return sorted(rng.choice(most, size=n, replace=False).tolist())


@pytest.mark.parametrize("kv,dim,pad", [(1, 64, 0), (2, 128, 0), (5, 64, 0), (3, 96, 8), (2, 20, 0), (1, 1, 0), (4, 256, 0), (2, 64, 3), (40, 128, 0)])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_commit(torch, kv, dim, pad, page):
    rng = np.random.default_rng(dim + page)
    for most, ctx in ((1, [0]), (5, [0, 3, 47, 100]), (64, [16, 1, 95])):
        n, layers = len(ctx), 3
        width = -(-(max(ctx) + most) // page)
        shape = (layers, n * width + 2, page, kv, dim)
        kc, vc = _cache(torch, shape, 1, pad=pad), _cache(torch, shape, 2, pad=pad)
        table = rng.permutation(n * width + 2)[:n * width].reshape(n, width).astype(np.int32)
        count = [int(rng.integers(0, most + 1)) for _ in ctx[:-1]] + [max(1, most // 2)]
        path = np.full((n, most), -1, np.int32)
        for s, c in enumerate(count):
            path[s, :c] = _path(rng, c, most)
        want = behind_ref.commit(_bits(torch, kc), _bits(torch, vc), table, ctx, path, count)
        out, err = Guarded(torch, (n,), torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
        dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        cbq.cbq_kv_commit(kc, vc, dev(table), dev(ctx), dev(path), dev(count), out=out.view, err=err)
        torch.cuda.synchronize()
        out.check()
        assert int(err) == 0 and list(out.view.cpu().numpy()) == [a + b for a, b in zip(ctx, count)]
        assert np.array_equal(_bits(torch, kc), want[0]) and np.array_equal(_bits(torch, vc), want[1])


def test_commit_of_one_layer_and_any_order_of_axes(torch):
    """A cache of four axes, heads before tokens in memory; layers inside pages."""
    for strides in ("heads", "layers"):
        x = [_cache(torch, (6, 2, 16, 64), i) if strides == "heads" else _cache(torch, (6, 3, 16, 2, 64), i) for i in (1, 2)]
        kc, vc = (t.transpose(1, 2) if strides == "heads" else t.transpose(0, 1) for t in x)
        five = [(_bits(torch, t)[None] if strides == "heads" else _bits(torch, t)) for t in (kc, vc)]
        table, ctx, path, count = np.array([[4, 1, 3]], np.int32), [14], np.array([[0, 2, 5, 9, -1]], np.int32), [4]
        path_dev = torch.from_numpy(np.pad(path, ((0, 0), (0, 7)), constant_values=-1)).cuda()
        want = behind_ref.commit(*five, table, ctx, path, count)
        dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        got = cbq.cbq_kv_commit(kc, vc, torch.from_numpy(table).cuda(), dev(ctx), path_dev, dev(count))
        assert got.tolist() == [18]
        for t, w in zip((kc, vc), want):
            b = _bits(torch, t)
            assert np.array_equal(b[None] if strides == "heads" else b, w)


def test_commit_of_bad_paths(torch):
    """What is wrong ends the sequence's moves there, and the others' go on."""
    page, most = 4, 6
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    # (path, count, ctx, table row, good entries, bits)
    ok = [0, 1, 2, 3, 4, 5]
    rows = [([0, 2, 4, -1, -1, -1], 3, 5, ok, 3, 0), ([0, 3, 3, 5, -1, -1], 4, 5, ok, 2, BAD_LENGTH),
            ([0, 2, 1, 5, -1, -1], 4, 5, ok, 2, BAD_LENGTH), ([1, 2, 6, 7, -1, -1], 4, 5, ok, 2, BAD_LENGTH),
            ([0, -1, 3, 5, -1, -1], 4, 5, ok, 1, BAD_LENGTH), ([0, 2, 3, 4, 5, 9], 9, 5, ok, 5, BAD_LENGTH),
            ([0, 2, 3, 4, 5, 9], -2, 5, ok, 0, BAD_LENGTH), ([0, 2, 3, -1, -1, -1], 3, -1, ok, 0, BAD_LENGTH),
            ([0, 1, 3, 5, -1, -1], 4, 20, ok, 3, BAD_LENGTH), ([0, 2, 4, 5, -1, -1], 4, 5, [0, 1, 30, 3, 4, 5], 4, BAD_SLOT),
            ([0, 2, 4, 5, -1, -1], 4, 5, [0, -1, 2, 3, 4, 5], 4, BAD_SLOT), ([1, 2, 3, 4, 5, -1], 5, 2 ** 31 - 3, ok, 0, BAD_LENGTH)]
    for i, (path, count, ctx, table, good, bits) in enumerate(rows):
        both = [rows[i], rows[0]]
        tables = np.array([table, [6, 7, 8, 9, 10, 11]], np.int32)
        kc, vc = _cache(torch, (2, 12, page, 2, 64), 1), _cache(torch, (2, 12, page, 2, 64), 2)
        before = _bits(torch, kc), _bits(torch, vc)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = cbq.cbq_kv_commit(kc, vc, torch.from_numpy(tables).cuda(), dev([r[2] for r in both]), dev([r[0] for r in both]),
                                dev([r[1] for r in both]), err=err)
        assert int(err) == bits and out.tolist() == [ctx + good, 8], i
        safe = [min(max(t, 0), 11) for t in table]
        moves = [(a, b) for a, b in enumerate(path[:good])
                 if all(0 <= table[(ctx + x) // page] < 12 for x in (a, b))] if good else []
        want = [x.copy() for x in before]
        for x, y in zip(want, before):
            for a, b in moves:
                x[:, safe[(ctx + a) // page], (ctx + a) % page] = y[:, safe[(ctx + b) // page], (ctx + b) % page]
            for a, b in enumerate([0, 2, 4]):
                x[:, tables[1][(5 + a) // page], (5 + a) % page] = y[:, tables[1][(5 + b) // page], (5 + b) % page]
        assert np.array_equal(_bits(torch, kc), want[0]) and np.array_equal(_bits(torch, vc), want[1]), i


def test_commit_refusals(torch):
    kc, vc = _cache(torch, (2, 4, 4, 2, 64), 1), _cache(torch, (2, 4, 4, 2, 64), 2)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [kc, vc, i(1, 2), i(1), i(1, 3), i(1)]
    cbq.cbq_kv_commit(*good)
    for at, x, e in ((1, vc[:1], ValueError), (0, kc.float(), TypeError), (2, i(2, 2), ValueError), (4, i(3), ValueError),
                     (4, i(1, 65), cbq.CbqError), (5, i(2), ValueError), (3, i(1).long(), TypeError)):
        args = list(good)
        args[at] = x
        with pytest.raises(e):
            cbq.cbq_kv_commit(*args)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_kv_commit(*good, out=good[3])


def _pages8(torch, layers, pages, page, kv, dim, block, pad=0):
    """An 8-bit cache and scales between guards, filled with a pattern."""
    if pad:
        k8, v8 = (torch.full((layers, pages, page, kv, dim + pad), 0x33, dtype=torch.uint8, device="cuda") for _ in "kv")
        g = []
        k8, v8 = k8[..., :dim], v8[..., :dim]
    else:
        g = [Guarded(torch, (layers, pages, page, kv, dim), torch.uint8) for _ in "kv"]
        k8, v8 = (x.view.fill_(0x33) for x in g)
    s = [Guarded(torch, (layers, pages, page // block, kv), torch.float32) for _ in "kv"]
    ks, vs = (x.view.fill_(3.0) for x in s)
    f8 = torch.float8_e4m3fn
    return (k8.view(f8) if not pad else k8.as_strided(k8.size(), k8.stride()).view(f8), v8.view(f8), ks, vs), g + s


@pytest.mark.parametrize("kv,dim,pad", [(1, 64, 0), (2, 128, 0), (3, 96, 8), (2, 20, 0), (1, 1, 0), (4, 256, 0), (2, 64, 3)])
@pytest.mark.parametrize("page,block", [(1, 1), (16, 16), (16, 1), (48, 16), (64, 64), (128, 128), (6, 3)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_quantize(torch, kv, dim, pad, page, block, dtype):
    layers, pages, pages8 = 2, 5, 6
    shape = (layers, pages, page, kv, dim)
    g = torch.Generator(device="cuda").manual_seed(dim + page)
    kc, vc = (torch.randn((*shape[:-1], dim + pad), generator=g, device="cuda").to(getattr(torch, dtype))[..., :dim] for _ in "kv")
    kc *= torch.exp2(torch.randint(-8, 8, (1, pages, 1, kv, 1), generator=g, device="cuda").float()).to(kc.dtype)
    vc[:, 1] = 0
    src, dst = np.array([4, 1, -1, 0, 2], np.int32), np.array([0, 5, 3, -2, 4], np.int32)
    (k8, v8, ks, vs), guards = _pages8(torch, layers, pages8, page, kv, dim, block, pad)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cbq.cbq_kv_quantize(kc, vc, torch.from_numpy(src).cuda(), k8, v8, ks, vs, torch.from_numpy(dst).cuda(), err=err)
    torch.cuda.synchronize()
    for b in guards:
        b.check()
    assert int(err) == 0
    for x, got, scales in ((kc, k8, ks), (vc, v8, vs)):
        got, scales = got.float().cpu().numpy(), scales.cpu().numpy()
        same = float(torch.tensor([0x33], dtype=torch.uint8).view(torch.float8_e4m3fn).float())
        want, want_s = np.full(got.shape, same), np.full(scales.shape, 3.0)
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                for layer in range(layers):
                    q, s = behind_ref.quantize(x[layer, a:a + 1].double().cpu().numpy(), block)
                    want[layer, b], want_s[layer, b] = q[0], s[0]
        assert np.array_equal(scales, want_s) and np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_quantize_of_every_number(torch, dtype):
    """All 16-bit patterns, so many to a block that each meets scales of all sizes; NaN and infinities become NaN."""
    t = getattr(torch, dtype)
    x = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32, device="cuda").to(torch.int16)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.cat([x, x[torch.randperm(1 << 16, generator=g, device="cuda")]]).view(t).view(16, 64, 2, 64)
    (k8, v8, ks, vs), _ = _pages8(torch, 1, 16, 64, 2, 64, 8)
    pages = torch.arange(16, dtype=torch.int32, device="cuda")
    cbq.cbq_kv_quantize(x, x, pages, k8[0], v8[0], ks[0], vs[0], pages)
    want, scale = behind_ref.quantize(x.double().cpu().numpy(), 8)
    assert np.array_equal(ks[0].double().cpu().numpy(), scale) and torch.equal(ks, vs)
    got = k8[0].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    assert np.isnan(want).any() and torch.equal(k8.view(torch.uint8), v8.view(torch.uint8))


def test_quantize_of_bad_pages(torch):
    kc, vc = _cache(torch, (4, 16, 2, 64), 1, "float16"), _cache(torch, (4, 16, 2, 64), 2, "float16")
    (k8, v8, ks, vs), guards = _pages8(torch, 1, 3, 16, 2, 64, 16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for src, dst in ((i(4), i(0)), (i(0), i(3)), (i(1 << 30), i(1 << 30)), (i(-1), i(3)), (i(4), i(-1))):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cbq.cbq_kv_quantize(kc, vc, src, k8[0], v8[0], ks[0], vs[0], dst, err=err)
        assert int(err) == BAD_SLOT
    for b in guards:
        b.check()
    assert bool((k8.view(torch.uint8) == 0x33).all()) and bool((ks == 3).all())


def test_quantize_refusals(torch):
    kc, vc = _cache(torch, (4, 16, 2, 64), 1), _cache(torch, (4, 16, 2, 64), 2)
    (k8, v8, ks, vs), _ = _pages8(torch, 1, 3, 16, 2, 64, 16)
    k8, v8, ks, vs = k8[0], v8[0], ks[0], vs[0]
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [kc, vc, i(0), k8, v8, ks, vs, i(0)]
    cbq.cbq_kv_quantize(*good)
    for at, x, e in ((2, i(0, 1), ValueError), (3, k8.view(torch.uint8), TypeError), (5, ks.half(), TypeError),
                     (4, v8[:2], ValueError), (5, ks[:2], ValueError), (2, i(0).long(), TypeError), (0, kc[..., :32], ValueError)):
        args = list(good)
        args[at] = x
        with pytest.raises(e):
            cbq.cbq_kv_quantize(*args)
    with pytest.raises(cbq.CbqError):  # pages of another size
        cbq.cbq_kv_quantize(kc[:, :8], vc[:, :8], *good[2:])
    with pytest.raises(ValueError):  # five scales to sixteen tokens
        cbq.cbq_kv_quantize(kc, vc, i(0), k8, v8, *(torch.ones((3, 5, 2), device="cuda") for _ in "kv"), i(0))
