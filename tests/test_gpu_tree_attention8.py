"""Attention of drafted trees over contexts whose older places are in 8 bits
(cbq_tree_attention8) on the GPU against the definition in 64 bits, with keys and
values that the 8-bit numbers and their scales stand for.

Tolerances are those of the 16-bit cache's (a score off by delta = (dim + 8)
2^-24 scale sum|q k|, a weight rounded to half a step of its type, fp32 sums),
and for old places: the query's rounding, 2^-38 of the row's largest for each
dim, which delta's constant holds; weights in fp16, whose half step is no more
than the 16-bit type's own, and below 2^-24 of the row's largest (weight times
scale) 2^-25 2^-10 of that absolutely, with numbers up to 448: keys 2^-35 448
max(scale) more.  The running maximum holds a scale's logarithm and 10, which
the lse gets back with 2^-23 of them."""
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


class Setup:
    """Sequences of old[i] places in 8 bits, recent[i] behind them and drafts[i] drafted tokens."""

    def __init__(self, torch, old, recent, drafts, heads, kv, dim, page=16, page8=None, block=16, dtype="bfloat16", seed=0,
                 sharp=1.0, spread=2, any_scale=False, pad=0, heads_first=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = getattr(torch, dtype)
        page8 = page if page8 is None else page8
        block = min(block, page8)
        self.torch, self.dt, self.page, self.page8, self.block = torch, dt, page, page8, block
        self.old, self.ctx = np.array(old, np.int32), np.array(old, np.int32) + np.array(recent, np.int32)
        self.start = np.cumsum([0] + list(drafts)).astype(np.int32)
        total, n = int(self.start[-1]), len(old)
        self.q = (torch.randn((total, heads, dim + pad), generator=g, device="cuda") * sharp).to(dt)[..., :dim]
        need8 = [-(-o // page8) for o in old]
        first = [o // page for o in old]
        need = [-(-int(c + d) // page) - f for c, d, f in zip(self.ctx, drafts, first)]

        def normal(pages, size):
            shape = (pages, kv, size, dim + pad) if heads_first else (pages, size, kv, dim + pad)
            x = torch.randn(shape, generator=g, device="cuda")
            return (x.transpose(1, 2) if heads_first else x)[..., :dim]

        pages8, pages = sum(need8) + 2, sum(need) + 2
        self.kc, self.vc = (normal(pages, page).to(dt) for _ in "kv")
        wide = 1 if pad == 0 else pad
        self.k8, self.v8 = (normal(pages8, page8).mul(100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in "kv")
        e = torch.randint(-spread, spread + 1, (2, pages8, page8 // block, kv * wide), generator=g, device="cuda").float()
        s = torch.exp2(e - 7)
        if any_scale:
            s *= 1 + torch.rand(s.shape, generator=g, device="cuda")
        self.ks, self.vs = s[0][..., ::wide], s[1][..., ::wide]
        ids8, ids = rng.permutation(pages8).astype(np.int32), rng.permutation(pages).astype(np.int32)
        self.table8 = np.full((n, max(1, max(need8))), -5, np.int32)  # what is past a sequence's places is not read
        self.table = np.full((n, max(1, max(f + w for f, w in zip(first, need)))), -7, np.int32)
        a = b = 0
        for i in range(n):
            self.table8[i, :need8[i]] = ids8[a:a + need8[i]]
            self.table[i, first[i]:first[i] + need[i]] = ids[b:b + need[i]]
            a, b = a + need8[i], b + need[i]
        self.mask = np.zeros(total, np.int64)
        for i, d in enumerate(drafts):
            for j in range(d):
                parent = rng.integers(-1, j) if j else -1
                bits = (int(self.mask[self.start[i] + parent]) if parent >= 0 else 0) | 1 << j
                self.mask[self.start[i] + j] = bits - (1 << 64) if bits >> 63 & 1 else bits
        self.limits = dict(max_tok=max(1, max(drafts)), max_old=max(old), max_new=max(1, max(r + d for r, d in zip(recent, drafts))))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self):
        t = lambda a: self.torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return (self.q, self.k8, self.v8, self.ks, self.vs, t(self.table8), t(self.old), self.kc, self.vc, t(self.table),
                t(self.ctx), t(self.start), t(self.mask))

    def run(self, **how):
        how = dict(dict(self.limits, with_lse=True, err=self.err), **how)
        return cbq.cbq_tree_attention8(*self.args(), **how)

    def seqs(self):
        """The sequences as the kernels may see them, within the call's limits."""
        n = lambda x: x.double().cpu().numpy()  # noqa: E731
        k8, v8, ks, vs, kc, vc = (n(x) for x in (self.k8, self.v8, self.ks, self.vs, self.kc, self.vc))
        out, lim = [], self.limits
        for i in range(len(self.old)):
            row0, rows = int(self.start[i]), int(min(self.start[i + 1] - self.start[i], lim["max_tok"]))
            ctx = max(0, int(self.ctx[i]))
            first = max(0, min(int(self.old[i]), ctx))
            last8 = min(first, lim["max_old"], self.table8.shape[1] * self.page8)
            most = max(first, min(first + lim["max_new"], self.table.shape[1] * self.page))
            end = min(ctx + rows, most)
            ctx = min(ctx, most)
            k, v, place = [], [], []
            for p in range(last8):
                page, t = int(self.table8[i][p // self.page8]), p % self.page8
                if 0 <= page < k8.shape[0]:
                    k.append(k8[page, t] * ks[page, t // self.block][:, None])
                    v.append(v8[page, t] * vs[page, t // self.block][:, None])
                    place.append(p)
            for p in range(first, end):
                page = int(self.table[i][p // self.page])
                if 0 <= page < kc.shape[0]:
                    k.append(kc[page, p % self.page])
                    v.append(vc[page, p % self.page])
                    place.append(p)
            kv, dim = kc.shape[2:]
            place = np.array(place, np.int64)
            seen = np.array([[p < ctx or bool(int(self.mask[row0 + r]) >> int(p - ctx) & 1) for p in place] for r in range(rows)],
                            bool).reshape(rows, len(place))
            out.append((row0, np.array(k).reshape(-1, kv, dim), np.array(v).reshape(-1, kv, dim), seen))
        return out

    def check(self, out, lse, scale=None, seqs=None):
        torch, dim = self.torch, self.q.shape[2]
        scale = dim ** -0.5 if scale is None else scale
        seqs = self.seqs() if seqs is None else seqs
        o, l, absv, big = behind_ref.attention(self.q.double().cpu().numpy(), seqs, scale)
        keys = max([1] + [s[1].shape[0] for s in seqs])
        delta = (dim + 8) * 2.0 ** -24 * big
        lim = absv * (torch.finfo(self.dt).eps / 2 + 4 * delta[..., None] + (keys + 32) * 2.0 ** -24)
        lim = lim + keys * 2.0 ** -35 * 448 * float(self.vs.max())
        if self.dt == torch.float16:
            lim = lim + keys * 2.0 ** -25 * 6
        if out.dtype != torch.float32:
            lim = lim + (np.abs(o) + lim) * torch.finfo(out.dtype).eps / 2 + (2.0 ** -25 if self.dt == torch.float16 else 0)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bad = ~(np.abs(got - o) <= lim)
        assert not bad.any(), f"out: {bad.sum()} off, first at {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - o) / (lim + 1e-30))}"
        none = np.isneginf(l)
        assert np.array_equal(none, np.isneginf(gl)) and np.all(got[none] == 0)
        far = np.abs(gl[~none] - l[~none])
        lv = float(torch.log2(self.vs).abs().max()) + 10
        assert np.all(far <= delta[~none] + 2.0 ** -22 + 2.0 ** -23 * (np.abs(l[~none]) + lv) + keys * 2.0 ** -24), far.max()


def _go(torch, *a, scale=None, **k):
    s = Setup(torch, *a, **k)
    g = Guarded(torch, s.q.shape, s.dt)
    out, lse = s.run(out=g.view, scale=scale)
    torch.cuda.synchronize()
    g.check()
    assert s.err.item() == 0
    s.check(out, lse, scale)
    return s


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (32, 8, 128), (16, 1, 128), (14, 2, 64), (6, 2, 256), (40, 1, 256), (24, 1, 256),
                                          (5, 5, 1), (4, 2, 80), (3, 1, 192), (4, 1, 67), (71, 1, 64)])
@pytest.mark.parametrize("old,recent,drafts", [([130], [0], [1]), ([0, 64, 200], [5, 3, 17], [5, 1, 17])])
def test_heads_and_dims(torch, dtype, heads, kv, dim, old, recent, drafts):
    _go(torch, old, recent, drafts, heads, kv, dim, dtype=dtype, seed=heads + dim)


@pytest.mark.parametrize("page,page8,block", [(1, 1, 1), (5, 15, 5), (16, 16, 1), (16, 64, 64), (48, 48, 16), (64, 16, 4), (128, 128, 128),
                                              (16, 1000, 8)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages_and_blocks(torch, page, page8, block, heads_first):
    """Pages of either cache that end inside a tile, scales for a token and for a page; both orders of memory."""
    for dtype, dim in (("bfloat16", 128), ("float16", 64)):
        _go(torch, [0, 1, 299, 64], [1, 0, 13, 70], [1, 3, 2, 6], 8, 2, dim, page, page8, block, dtype, seed=page, heads_first=heads_first)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths(torch, n):
    """Old places, and those behind, around every border of a tile, alone and in a batch."""
    _go(torch, [n], [0], [1], 8, 2, 128, seed=n)
    _go(torch, [64], [n], [1], 8, 2, 128, seed=n)
    _go(torch, [n, 700, max(0, n - 3)], [5, n, 0], [4, 2, 3], 4, 2, 64, 32, seed=n, dtype="float16")


@pytest.mark.parametrize("drafts", [[1], [3], [8], [16], [17], [32], [33], [64], [64, 0, 1, 0, 40]])
@pytest.mark.parametrize("heads,kv,dim", [(4, 1, 64), (8, 1, 128), (3, 3, 64), (14, 2, 128), (4, 2, 256)])
def test_trees(torch, drafts, heads, kv, dim):
    old = [100, 33, 0, 5, 1][:len(drafts)]
    _go(torch, old, [20, 0, 3, 1, 0][:len(drafts)], drafts, heads, kv, dim, seed=sum(drafts) + heads)


@pytest.mark.parametrize("old,recent", [(4096, 100), (20000, 0), (3000, 3000)])
@pytest.mark.parametrize("heads,kv,drafts", [(8, 8, 1), (32, 8, 5), (16, 1, 16), (8, 1, 64)])
def test_long(torch, old, recent, heads, kv, drafts):
    """Long enough that the keys of one row are split and joined, sequences that need few of the parts among them."""
    _go(torch, [old, 7, 0, old // 3], [recent, 0, recent, 9], [drafts, 1, drafts, drafts], heads, kv, 128, 64, seed=old)


@pytest.mark.parametrize("heads,drafts,dim", [(8, 4, 128), (8, 40, 128), (8, 40, 64), (4, 4, 256), (4, 4, 72)])
def test_scales(torch, heads, drafts, dim):
    """Scales far apart from block to block, and of any value; scores far apart, equal, and turned round."""
    a = [900, 40], [30, 2], [drafts, 1], heads, 2, dim
    _go(torch, *a, seed=1, spread=20, block=4, sharp=0.01)
    _go(torch, *a, seed=2, spread=3, block=4, any_scale=True)
    _go(torch, *a, seed=3, sharp=8.0)
    _go(torch, *a, seed=4, scale=0.0)
    _go(torch, *a, seed=5, scale=-0.1)
    _go(torch, *a, seed=6, dtype="float16", spread=12, block=1, sharp=0.1, any_scale=True)


def test_ends_of_the_scales(torch):
    """All values tiny or huge: results in fp32, relative to their size."""
    for e in (-80, 112):
        s = Setup(torch, [500], [0], [3], 4, 2, 128, seed=e + 80)
        s.vs = torch.full_like(s.vs, 2.0 ** e)
        s.vc = torch.zeros_like(s.vc)
        s.vc[:] = 2.0 ** e if e > 0 else 0.0
        out = torch.empty(s.q.shape, device="cuda")
        out, lse = s.run(out=out)
        s.check(out, lse)
        assert float(out.abs().max()) > 2.0 ** e


def test_small_and_large_queries(torch):
    """Rows of a query of every size its type has; scores stay moderate through the scale."""
    for f, scale in ((2.0 ** -100, 2.0 ** 98), (2.0 ** 60, 2.0 ** -62), (2.0 ** -126, 1.0), (0.0, 1.0)):
        s = Setup(torch, [300], [0], [4], 4, 2, 64, seed=3)
        s.q = (s.q.float() * f).bfloat16()
        s.kc = torch.zeros_like(s.kc)
        out, lse = s.run(scale=scale)
        s.check(out, lse, scale)


def test_strides(torch):
    """A query, both caches and scales inside wider tensors: by 16 bytes, and not."""
    for pad in (16, 8, 3):
        for dim in (64, 128):
            _go(torch, [200, 0, 70], [3, 9, 0], [3, 1, 7], 8, 2, dim, 16, 32, 8, seed=pad, pad=pad)


def test_results_in_32_bits(torch):
    for dtype in ("bfloat16", "float16"):
        for drafts in (3, 50):
            s = Setup(torch, [700, 9], [40, 5], [drafts, 2], 8, 2, 128, dtype=dtype, seed=4)
            out, lse = s.run(out=torch.empty(s.q.shape, device="cuda"))
            assert out.dtype == torch.float32
            s.check(out, lse)


def test_no_old_places(torch):
    """max_old = 0: the 16-bit cache's attention."""
    for ctx, drafts, heads, kv, dim in (([0, 300], [1, 5], 8, 2, 128), ([5000], [4], 16, 2, 64), ([900], [40], 8, 1, 128), ([30], [2], 2, 2, 40)):
        s = Setup(torch, [0] * len(ctx), ctx, drafts, heads, kv, dim, seed=5)
        assert s.limits["max_old"] == 0
        out, lse = s.run()
        s.check(out, lse)
        t = s.args()
        want, want_lse = cbq.cbq_tree_attention(s.q, s.kc, s.vc, *t[9:], max_tok=s.limits["max_tok"], max_len=s.limits["max_new"], with_lse=True)
        s.check(want, want_lse)


def test_rows_that_see_nothing(torch):
    for dim in (128, 64, 40):
        for old, recent in ((0, 0), (40, 3)):
            s = Setup(torch, [old, 9], [recent, 1], [5, 3], 4, 2, dim, seed=6)
            s.mask[:5] = [0, 1, 0, 2, 0]
            out, lse = s.run()
            s.check(out, lse)
            assert (old > 0) == bool(torch.isfinite(lse[0]).all())


PATHS = {"a warp a row": ([200], [40], [3], 4, 2, 80), "one block each": ([60], [5], [3], 4, 2, 64), "64 rows": ([60], [5], [20], 3, 1, 64),
         "a cluster": ([300], [20], [1], 32, 8, 128), "heads of 256": ([250], [30], [5], 6, 2, 256),
         "parts": ([8192], [100], [5], 32, 8, 128), "a batch": ([2000] * 24, [40] * 24, [5] * 24, 32, 8, 128),
         "many rows": ([70] * 40, [9] * 40, [40] * 40, 16, 4, 128), "many rows, parts": ([3000], [50], [40], 8, 1, 128),
         "many rows, heads of 64": ([9000, 300], [20, 1], [40, 3], 16, 2, 64)}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_nan(torch, path, dtype):
    """NaN in a query is its row's; in an old key, value or scale its kv head's; in a draft that a row does not see, no one's."""
    old, recent, drafts, heads, kv, dim = PATHS[path]
    s = Setup(torch, old, recent, drafts, heads, kv, dim, dtype=dtype, seed=dim)
    whole, lse = s.run()
    q = s.q.clone()
    row, head = len(s.mask) - 1, heads - 1
    s.q[row, head, 7:8] = float("nan")
    out, lse2 = s.run()
    odd = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    odd[row, head] = True
    assert torch.isnan(out[odd]).all() and torch.isnan(lse2[odd]).all()
    assert torch.equal(out[~odd], whole[~odd]) and torch.equal(lse2[~odd], lse[~odd])
    s.q = q
    i, p = len(old) - 1, old[-1] - 1
    rows, h = slice(int(s.start[i]), int(s.start[i + 1])), slice((kv - 1) * (heads // kv), heads)
    page, t = int(s.table8[i][p // s.page8]), p % s.page8
    odd = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    odd[rows, h] = True
    for name in ("k8", "v8", "ks", "vs"):
        x = getattr(s, name)
        kept = x.clone()
        if name[1] == "8":
            x.view(torch.uint8)[page, t, kv - 1, 3] = 0x7F
        else:
            x[page, t // s.block, kv - 1] = float("nan")
        out, lse2 = s.run()
        setattr(s, name, kept)
        bad = torch.isnan(out).any(-1)
        if name[0] == "k" or name == "vs":
            assert torch.isnan(out[odd]).all(), name
        else:
            assert torch.isnan(out[odd][..., 3]).all(), name
        assert not bad[~odd].any() and torch.equal(out[~odd], whole[~odd]) and torch.equal(lse2[~odd], lse[~odd]), name
    # a draft's key and value with NaN and infinity: for the rows that see it
    d = int(s.start[-1] - s.start[-2]) - 1
    page, t = int(s.table[i][(s.ctx[i] + d) // s.page]), int((s.ctx[i] + d) % s.page)
    s.vc[page, t, kv - 1, 2], s.kc[page, t, kv - 1, 1] = float("inf"), float("nan")
    out, lse2 = s.run()
    sees = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    for r in range(int(s.start[i]), int(s.start[i + 1])):
        sees[r, h] = bool(int(s.mask[r]) >> d & 1)
    assert torch.isnan(out[sees]).all() and torch.equal(out[~sees], whole[~sees]) and torch.equal(lse2[~sees], lse[~sees])
    assert s.err.item() == 0


@pytest.mark.parametrize("dim", [128, 64, 48])
@pytest.mark.parametrize("drafts", [3, 40])
def test_pages_that_do_not_exist(torch, dim, drafts):
    """Their keys are seen by nobody, and the call says so."""
    s = Setup(torch, [200, 300], [40, 20], [drafts, 2], 8, 2, dim, seed=7)
    s.table8[0, 3], s.table8[1, 0], s.table8[1, 18] = -1, 10 ** 6, s.k8.shape[0]
    s.table[0, 14] = s.kc.shape[0]
    out, lse = s.run()
    assert s.err.item() == BAD_SLOT
    s.check(out, lse)


@pytest.mark.parametrize("dim", [128, 64, 48])
@pytest.mark.parametrize("drafts", [3, 40])
def test_lengths_that_do_not_fit(torch, dim, drafts):
    """Old places beyond max_old or the table, recent ones beyond max_new or the table, old ones beyond the context."""
    def go(change):
        s = Setup(torch, [200, 300], [40, 20], [drafts, 2], 8, 2, dim, seed=8)
        change(s)
        out, lse = s.run()
        assert s.err.item() == BAD_LENGTH
        s.check(out, lse)

    go(lambda s: s.limits.update(max_old=290))
    go(lambda s: s.limits.update(max_old=0))
    go(lambda s: s.limits.update(max_new=22))
    go(lambda s: s.limits.update(max_new=1))
    go(lambda s: setattr(s, "table8", s.table8[:, :17]))
    go(lambda s: setattr(s, "table", s.table[:, :20]))
    go(lambda s: setattr(s, "table", s.table[:, :13]))
    s = Setup(torch, [200, 300], [40, 20], [drafts, 2], 8, 2, dim, seed=8)
    s.limits.update(max_tok=2)
    out, lse = s.run(out=torch.full_like(s.q, 7.0))
    assert s.err.item() == BAD_LENGTH and bool((out[2:drafts] == 7).all())  # rows behind the cut stay as they were
    out[2:drafts], lse[2:drafts] = 0, -float("inf")
    s.check(out, lse)
    s = Setup(torch, [200, 300], [40, 20], [drafts, 2], 8, 2, dim, seed=8)
    s.old[0] = -3  # none old: the places in front are not in the table
    s.table[0] = np.arange(s.table.shape[1]) % s.kc.shape[0]
    s.limits["max_new"] = 300
    out, lse = s.run()
    assert s.err.item() == BAD_LENGTH
    s.check(out, lse)
    s.old[0] = 900  # beyond the context: all 240 places of it are old, for the last 32 of which the table has no pages
    out, lse = s.run()
    assert s.err.item() == BAD_LENGTH | BAD_SLOT
    s.check(out, lse)


def test_workspace_and_refusals(torch):
    s = Setup(torch, [6000], [40], [3], 32, 8, 128, seed=9)
    lim = s.limits
    room = cbq.cbq_tree_attention8_workspace(1, 3, lim["max_tok"], lim["max_old"], lim["max_new"], 32, 8, 128)
    assert room > 16
    g = Guarded(torch, (room,), torch.uint8)
    out, lse = s.run(workspace=g.view)
    g.check()
    s.check(out, lse)
    with pytest.raises(cbq.CbqError):
        s.run(workspace=g.view[:-16])
    for how in (dict(max_old=-1), dict(max_new=0), dict(max_tok=0), dict(max_old=1 << 30)):
        with pytest.raises(cbq.CbqError):
            s.run(**how)
    a = list(s.args())
    for at, x, e in ((1, s.k8.view(torch.uint8), TypeError), (3, s.ks.half(), TypeError), (2, s.v8[:3], ValueError),
                     (5, a[5][0], ValueError), (6, a[6].long(), TypeError), (0, s.q.float(), ValueError),
                     (0, s.q[..., :64], ValueError), (7, s.kc[:2], ValueError)):
        args = list(a)
        args[at] = x
        with pytest.raises(e):
            cbq.cbq_tree_attention8(*args, **lim)
