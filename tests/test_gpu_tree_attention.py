"""Attention of drafted trees over a paged cache (cbq_tree_attention) on the
GPU against the definition in 64 bits.

Tolerances.  A score is a sum of dim products in fp32: off by at most delta =
(dim + 8) 2^-24 scale sum|q k| in the exponent (with the scaling and the
exponential's own 4 ulp in the constant), so a weight is off by a factor 1 +-
2 delta relative to the sum, and by half a step of the 16-bit type for the
product with v; sums and divisions in fp32 add (keys + 32) 2^-24.  Against
sum w|v| = A: |out - want| <= A (eps/2 + 4 delta + (keys + 32) 2^-24), and
half a step of the output type.  fp16 weights below 2^-14 of the row's top
lose 2^-25 absolutely: keys 2^-25 max|v| more.  lse is off by delta + 2^-22 +
2^-23 |lse| + keys 2^-24."""
import numpy as np
import pytest

from tests import step_ref
from tests.gpu_util import Guarded, cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


class Setup:
    """Random sequences: ctx[i] committed and drafts[i] drafted tokens each."""

    def __init__(self, torch, ctx, drafts, heads, kv, dim, page, dtype="bfloat16", seed=0, heads_first=False,
                 extra_width=0, sharp=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = getattr(torch, dtype)
        self.torch, self.dt, self.page = torch, dt, page
        self.ctx, self.start = np.array(ctx), np.cumsum([0] + list(drafts))
        need = [-(-(c + n) // page) for c, n in zip(ctx, drafts)]
        pages = sum(need) + 3
        total = int(self.start[-1])
        self.q = (torch.randn((total, heads, dim), generator=g, device="cuda") * sharp).to(dt)
        shape = (pages, kv, page, dim) if heads_first else (pages, page, kv, dim)
        self.kc, self.vc = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in "kv")
        if heads_first:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        ids = rng.permutation(pages)
        self.spare = ids[sum(need):]
        self.table = np.full((len(ctx), max(1, max(need)) + extra_width), self.spare[0], dtype=np.int32)
        at = 0
        for i, w in enumerate(need):
            self.table[i, :w] = ids[at:at + w]
            at += w
        self.mask = np.zeros(total, dtype=np.int64)
        for i, n in enumerate(drafts):
            for j in range(n):
                parent = rng.integers(-1, j) if j else -1
                bits = (int(self.mask[self.start[i] + parent]) if parent >= 0 else 0) | 1 << j
                self.mask[self.start[i] + j] = bits - (1 << 64) if bits >> 63 & 1 else bits
        self.max_tok, self.max_len = max(1, max(drafts)), max(1, max(c + n for c, n in zip(ctx, drafts)))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self):
        t = lambda a, d: self.torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731
        i32 = self.torch.int32
        return t(self.table, i32), t(self.ctx, i32), t(self.start, i32), t(self.mask, self.torch.int64)

    def run(self, out=None, **how):
        how = dict(dict(max_tok=self.max_tok, max_len=self.max_len), **how)
        return cbq.cbq_tree_attention(self.q, self.kc, self.vc, *self.dev(), with_lse=True, out=out, err=self.err, **how)

    def want(self, scale):
        n = lambda x: x.double().cpu().numpy()  # noqa: E731
        return step_ref.attention(n(self.q), n(self.kc), n(self.vc), self.table, self.ctx, self.start, self.mask, scale)

    def check(self, out, lse, scale=None, want=None):
        torch, dim = self.torch, self.q.shape[2]
        scale = dim ** -0.5 if scale is None else scale
        o, l, absv, big = want or self.want(scale)
        keys = max(1, int(np.max(self.ctx + np.diff(self.start))))
        delta = (dim + 8) * 2.0 ** -24 * big
        lim = absv * (torch.finfo(self.dt).eps / 2 + 4 * delta[..., None] + (keys + 32) * 2.0 ** -24)
        if self.dt == torch.float16:
            lim = lim + keys * 2.0 ** -25 * 6
        if out.dtype != torch.float32:
            lim = lim + (np.abs(o) + lim) * torch.finfo(out.dtype).eps / 2 + (2.0 ** -25 if self.dt == torch.float16 else 0)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bad = ~(np.abs(got - o) <= lim)
        assert not bad.any(), f"out: {bad.sum()} off, first at {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - o) / (lim + 1e-30))}"
        none = np.isneginf(l)
        assert np.array_equal(none, np.isneginf(gl))
        assert np.all(got[none] == 0)
        far = np.abs(gl[~none] - l[~none])
        assert np.all(far <= delta[~none] + 2.0 ** -22 + 2.0 ** -23 * np.abs(l[~none]) + keys * 2.0 ** -24), far.max()


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
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (32, 8, 128), (8, 8, 128), (16, 1, 128), (14, 2, 64), (6, 2, 256),
                                          (5, 5, 1), (4, 2, 80), (2, 1, 96), (3, 1, 192), (4, 1, 67), (71, 1, 64)])
@pytest.mark.parametrize("ctx,drafts", [([130], [1]), ([0, 63, 200], [5, 1, 17])])
def test_heads_and_dims(torch, dtype, heads, kv, dim, ctx, drafts):
    _go(torch, ctx, drafts, heads, kv, dim, 16, dtype=dtype, seed=heads + dim)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 64, 128, 1000])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(torch, page, heads_first):
    """Pages that end inside a tile, single tokens, one page for all; both orders of memory."""
    _go(torch, [0, 1, 299, 64], [1, 3, 2, 6], 8, 2, 128, page, seed=page, heads_first=heads_first, extra_width=2)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 95, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths(torch, n):
    """Lengths around every border of a tile, alone and in a batch."""
    _go(torch, [n], [1], 8, 2, 128, 16, seed=n)
    _go(torch, [n, 700, max(0, n - 3)], [4, 2, 3], 4, 2, 64, 32, seed=n, dtype="float16")


@pytest.mark.parametrize("drafts", [[1], [2], [3], [8], [9], [16], [31], [32], [33], [63], [64], [64, 0, 1, 0, 40]])
@pytest.mark.parametrize("heads,kv", [(4, 1), (8, 1), (3, 3), (14, 2)])
def test_trees(torch, drafts, heads, kv):
    """Trees up to 64 drafts, sequences without drafts among them."""
    ctx = [100, 33, 0, 5, 1][:len(drafts)]
    _go(torch, ctx, drafts, heads, kv, 64, 16, seed=sum(drafts) + heads)


@pytest.mark.parametrize("ctx", [4095, 20000])
@pytest.mark.parametrize("heads,kv,drafts", [(8, 8, 1), (32, 8, 5), (16, 1, 16), (8, 1, 64)])
def test_long(torch, ctx, heads, kv, drafts):
    """Long enough that the keys of one row are split and joined."""
    _go(torch, [ctx, 7, ctx // 3], [drafts, 1, drafts], heads, kv, 128, 64, seed=ctx)


def test_sharp_and_flat_scores(torch):
    """Scores far apart (the top moves along the keys), and no scale at all (plain means)."""
    _go(torch, [900], [4], 8, 2, 128, 16, seed=1, sharp=8.0)
    _go(torch, [900], [4], 8, 2, 128, 16, seed=2, scale=0.0)
    _go(torch, [900], [4], 8, 2, 128, 16, seed=3, scale=-0.1)


def test_rows_that_see_nothing(torch):
    """No committed token and an empty mask: zeros and -inf, beside rows that see something."""
    s = Setup(torch, [0, 0, 40], [3, 2, 3], 8, 2, 64, 16)
    s.mask[:] = [0, 2, 0, 0, 0, 0, 1, 7]
    out, lse = s.run()
    s.check(out, lse)
    assert np.isneginf(lse.cpu().numpy()[[0, 2, 3, 4]]).all()


def test_bits_of_other_sequences_and_beyond(torch):
    """Bits at and above a sequence's own drafts name nothing."""
    s = Setup(torch, [40, 3], [3, 2], 8, 2, 64, 16)
    out, lse = s.run()
    own = s.mask.copy()
    s.mask = np.concatenate([own[:3] | ~7, own[3:] | ~3])
    out2, lse2 = s.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("odd", [float("nan"), float("inf"), -float("inf"), "lowest"])
@pytest.mark.parametrize("drafts,heads,kv,dim", [([5, 9], 8, 2, 64), ([5, 9], 8, 2, 128), ([33, 64], 16, 2, 128), ([2, 1], 4, 1, 80)])
def test_what_a_row_does_not_see(torch, odd, drafts, heads, kv, dim):
    """NaN, infinities and the type's lowest value in spare pages, behind the
    last token of a page and in drafts that a row does not see."""
    s = Setup(torch, [50, 130], drafts, heads, kv, dim, 16, extra_width=1)
    bad = torch.finfo(s.dt).min if odd == "lowest" else odd
    want = s.want(dim ** -0.5)
    used = np.zeros(s.kc.shape[:2], dtype=bool)
    for i in range(2):
        p = np.arange(s.ctx[i] + drafts[i])
        used[s.table[i][p // 16], p % 16] = True
    for c in (s.kc, s.vc):
        c[torch.from_numpy(~used).cuda()] = bad
    s.check(*s.run(), want=want)
    # one draft of each sequence that (but for itself and its descendants) no row sees
    for i in range(2):
        j = drafts[i] // 2
        p = s.ctx[i] + j
        for c in (s.kc, s.vc):
            c[int(s.table[i][p // 16]), int(p % 16)] = bad
    seen = np.array([bool(int(s.mask[r]) >> (drafts[i] // 2) & 1) for i in range(2) for r in range(s.start[i], s.start[i + 1])])
    out, lse = s.run()
    keep = torch.from_numpy(~seen).cuda()
    out2, lse2 = out.clone(), lse.clone()
    o, l = (torch.from_numpy(x).cuda() for x in want[:2])
    out2[~keep], lse2[~keep] = o[~keep].to(out.dtype), l[~keep].float()
    s.check(out2, lse2, want=want)
    if odd != "lowest":
        assert not torch.isfinite(out[~keep]).all(dim=-1).any()


def test_bad_pages_and_lengths_are_reported(torch):
    """A page outside the cache is not seen; what is beyond the limits is cut."""
    s = Setup(torch, [60, 40], [2, 2], 4, 2, 64, 16)
    keep = s.table.copy()
    for bad in (-1, s.kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        s.table = keep.copy()
        s.table[0, 1] = bad
        s.err.zero_()
        out, lse = s.run()
        assert s.err.item() == cbq.CBQ_DEVERR_BAD_SLOT
        # the same with those sixteen keys moved out: the first sequence's other pages, one page shorter
        s2 = Setup(torch, [60, 40], [2, 2], 4, 2, 64, 16)
        s2.table = np.concatenate([keep[:, :1], keep[:, 2:], keep[:, :1]], 1)
        s2.table[1] = keep[1]
        s2.ctx = np.array([44, 40])
        s2.check(out, lse)
    s.table = keep
    whole = s.run()
    for how, bit in ((dict(max_len=50), True), (dict(max_tok=1), True), (dict(max_len=62), False)):
        s.err.zero_()
        out, lse = s.run(**how)
        assert s.err.item() == (cbq.CBQ_DEVERR_BAD_LENGTH if bit else 0)
    assert torch.equal(out, whole[0])
    s.err.zero_()
    s.ctx = np.array([1000, -3])
    s.run()
    torch.cuda.synchronize()
    assert s.err.item() == cbq.CBQ_DEVERR_BAD_LENGTH
    s.ctx, s.start = np.array([60, 40]), np.array([0, 2, 70])
    s.err.zero_()
    out, lse = s.run()
    assert s.err.item() == cbq.CBQ_DEVERR_BAD_LENGTH
    s.start = np.array([3, 1, 4])
    s.err.zero_()
    s.run()
    torch.cuda.synchronize()
    assert s.err.item() == cbq.CBQ_DEVERR_BAD_LENGTH


def test_strided_queries_and_fp32_output(torch):
    s = Setup(torch, [300, 20], [5, 3], 8, 2, 128, 16)
    wide = torch.zeros((8, 12, 136), dtype=s.dt, device="cuda")
    wide[:, 2:10, 3:131] = s.q
    whole, lse = s.run()
    s.q = wide[:, 2:10, 3:131]
    out, lse2 = s.run()
    assert torch.equal(out, whole) and torch.equal(lse, lse2)
    f = torch.empty(whole.shape, dtype=torch.float32, device="cuda")
    out, _ = s.run(out=f)
    s.check(out, lse)
    assert torch.equal(out.to(s.dt), whole)


def test_far_offsets(torch):
    """Pages beyond 2^31 values of the cache."""
    page, kv, dim = 64, 8, 128
    pages = (1 << 31) // (page * kv * dim) + 40
    kc, vc = (torch.empty((pages, page, kv, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    s = Setup(torch, [500], [4], 16, kv, dim, page)
    n = s.kc.shape[0]
    kc[-n:], vc[-n:] = s.kc, s.vc
    out, lse = s.run()
    s.kc, s.vc, s.table = kc, vc, s.table + (pages - n)
    out2, lse2 = s.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_repeat_stream_graph_and_refusals(torch):
    s = Setup(torch, [5000, 77], [5, 9], 32, 8, 128, 16)
    out, lse = s.run()
    for _ in range(3):
        again, lse2 = s.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    args = s.dev()
    ws = torch.full((cbq.cbq_tree_attention_workspace(2, 14, 9, s.max_len, 32, 8, 128),), 255, dtype=torch.uint8, device="cuda")
    into = torch.zeros_like(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cbq.cbq_tree_attention(s.q, s.kc, s.vc, *args, max_tok=9, max_len=s.max_len, out=into, workspace=ws)
    for _ in range(2):
        into.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, into)
    with pytest.raises(ValueError):
        cbq.cbq_tree_attention(s.q.half(), s.kc, s.vc, *args, max_tok=9, max_len=5009)
    with pytest.raises(TypeError):
        cbq.cbq_tree_attention(s.q, s.kc, s.vc, args[0].long(), *args[1:], max_tok=9, max_len=5009)
    with pytest.raises(ValueError):
        cbq.cbq_tree_attention(s.q, s.kc, s.vc, *args[:3], args[3][:2], max_tok=9, max_len=5009)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_tree_attention(s.q, s.kc, s.vc, *args, max_tok=65, max_len=5009)
    with pytest.raises(cbq.CbqError):
        cbq.cbq_tree_attention(s.q, s.kc, s.vc, *args, max_tok=9, max_len=5009, workspace=ws[:8])
