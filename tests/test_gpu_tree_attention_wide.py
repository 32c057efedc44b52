"""Many rows a kv head over long contexts (cbq_tree_attention's wide kernel for
the committed keys, joined with the drafts'), against the definition in 64
bits, with the tolerances of test_gpu_tree_attention: its row maximum may lag
by 2^8 (fp16: 2^5), which the last division takes out, so they hold as they
are."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_tree_attention import Setup, _go
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv,drafts", [(9, 1, 8), (16, 2, 16), (16, 2, 17), (6, 2, 43), (8, 1, 64), (14, 2, 37)])
def test_rows(torch, dtype, dim, heads, kv, drafts):
    """65 rows up to 512: one group of 128, two, two tiles of 256, ragged ones."""
    _go(torch, [1500], [drafts], heads, kv, dim, 16, dtype=dtype, seed=drafts + dim)


@pytest.mark.parametrize("ctx", [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 320, 1000, 1023, 1024, 1025])
@pytest.mark.parametrize("drafts", [9, 40])
def test_committed_lengths(torch, ctx, drafts):
    """Few tiles, an odd number of them, ragged ends; beside a long sequence and one without context."""
    _go(torch, [ctx, 1200, 0], [drafts, 3, drafts], 8, 1, 128, 48, seed=ctx)


@pytest.mark.parametrize("page", [1, 7, 64, 5000])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(torch, page, heads_first):
    _go(torch, [1100, 77], [12, 10], 16, 2, 128, page, seed=page, heads_first=heads_first)


@pytest.mark.parametrize("ctx,drafts", [([9000], [16]), ([30000], [33]), ([5000, 2000, 9000], [64, 1, 0])])
def test_chunks(torch, ctx, drafts):
    """Contexts that are split over blocks and joined."""
    _go(torch, ctx, drafts, 8, 1, 128, 64, seed=len(ctx))
    _go(torch, ctx, drafts, 8, 1, 64, 64, seed=len(ctx), dtype="float16")


def test_scores(torch):
    """Maxima that move along the keys (past the lag, and within it), a negative scale, and none."""
    for sharp in (0.1, 4.0, 12.0):
        _go(torch, [3000], [16], 8, 1, 128, 16, seed=int(sharp), sharp=sharp)
        _go(torch, [3000], [16], 8, 1, 128, 16, seed=int(sharp), sharp=sharp, dtype="float16")
    _go(torch, [2000], [16], 8, 1, 128, 16, seed=5, scale=-0.05)
    _go(torch, [2000], [16], 8, 1, 128, 16, seed=6, scale=0.0)
    s = Setup(torch, [4000], [16], 8, 1, 128, 16, seed=7)
    order = torch.from_numpy(s.table[0].astype(np.int64)).cuda()
    s.kc[order] *= torch.linspace(0.01, 3.0, len(order), device="cuda").to(s.dt)[:, None, None, None]
    s.check(*s.run())


@pytest.mark.parametrize("odd", [float("nan"), float("inf"), "lowest"])
def test_what_a_row_does_not_see(torch, odd):
    """Spare pages, the places behind the last token and unseen drafts."""
    s = Setup(torch, [1030, 70], [16, 12], 8, 1, 128, 48, extra_width=1)
    bad = torch.finfo(s.dt).min if odd == "lowest" else odd
    want = s.want(128 ** -0.5)
    used = np.zeros(s.kc.shape[:2], dtype=bool)
    for i, n in enumerate((16, 12)):
        p = np.arange(s.ctx[i] + n)
        used[s.table[i][p // 48], p % 48] = True
    for c in (s.kc, s.vc):
        c[torch.from_numpy(~used).cuda()] = bad
    s.check(*s.run(), want=want)
    p = s.ctx[0] + 8  # a draft of the first sequence
    for c in (s.kc, s.vc):
        c[int(s.table[0][p // 48]), int(p % 48)] = bad
    sees = np.array([bool(int(s.mask[r]) >> 8 & 1) for r in range(16)] + [False] * 12)
    out, lse = s.run()
    keep = torch.from_numpy(sees).cuda()
    out[keep], lse[keep] = torch.from_numpy(want[0]).cuda()[keep].to(out.dtype), torch.from_numpy(want[1]).cuda()[keep].float()
    s.check(out, lse, want=want)


def test_empty_rows(torch):
    """No committed token and an empty mask, in a batch whose others are long."""
    s = Setup(torch, [0, 2000], [10, 10], 8, 1, 128, 16)
    s.mask[:5] = 0
    out, lse = s.run()
    s.check(out, lse)
    assert np.isneginf(lse[:5].cpu().numpy()).all() and not out[:5].any()


def test_bad_pages_and_lengths(torch):
    s = Setup(torch, [2000, 40], [16, 2], 8, 1, 128, 16)
    keep = s.table.copy()
    whole = s.run()
    for bad in (-1, s.kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        s.table = keep.copy()
        s.table[0, 50] = bad
        s.err.zero_()
        out, lse = s.run()
        assert s.err.item() == cbq.CBQ_DEVERR_BAD_SLOT
        s2 = Setup(torch, [2000, 40], [16, 2], 8, 1, 128, 16)
        s2.table = np.delete(keep, 50, axis=1)
        s2.table[1, :3] = keep[1, :3]
        s2.ctx = np.array([1984, 40])
        s2.check(out, lse)
    s.table = keep
    for how, bit in ((dict(max_len=1500), True), (dict(max_tok=12), True), (dict(max_len=5000), False)):
        s.err.zero_()
        out, lse = s.run(**how)
        torch.cuda.synchronize()
        assert s.err.item() == (cbq.CBQ_DEVERR_BAD_LENGTH if bit else 0)
    s.check(out, lse)
    s.ctx = np.array([10 ** 6, -3])
    s.err.zero_()
    s.run()
    torch.cuda.synchronize()
    assert s.err.item() == cbq.CBQ_DEVERR_BAD_LENGTH


def test_strides_output_type_repeats_and_graph(torch):
    s = Setup(torch, [6000, 300], [20, 9], 16, 2, 128, 16)
    whole, lse = s.run()
    for _ in range(3):
        out, lse2 = s.run()
        assert torch.equal(out, whole) and torch.equal(lse, lse2)
    f = torch.empty(whole.shape, dtype=torch.float32, device="cuda")
    out, _ = s.run(out=f)
    assert torch.equal(out.to(s.dt), whole)
    wide = torch.zeros((29, 20, 136), dtype=s.dt, device="cuda")
    wide[:, 2:18, 3:131] = s.q
    s.q = wide[:, 2:18, 3:131]
    out, lse2 = s.run()
    assert torch.equal(out, whole) and torch.equal(lse, lse2)
    args = s.dev()
    into = torch.zeros_like(whole)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for _ in range(3):
            cbq.cbq_tree_attention(s.q, s.kc, s.vc, *args, max_tok=20, max_len=s.max_len, out=into)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(into, whole)


@pytest.mark.parametrize("drafts", [16, 32])
def test_rows_that_scale_alone(torch, drafts):
    """Along these keys the maxima of one warp's 32 rows grow at every tile, so
    that warp rescales its results each time while the others never do."""
    s = Setup(torch, [6000], [drafts], 8, 1, 128, 64, seed=3)
    s.q[4:] *= 0.001
    s.q[:4] = s.q[:4].abs() * 2
    order = torch.from_numpy(s.table[0].astype(np.int64)).cuda()
    s.kc[order] = (s.kc[order].abs().float() * torch.linspace(0.01, 3.0, len(order), device="cuda")[:, None, None, None]).to(s.dt)
    want = s.want(128 ** -0.5)
    for _ in range(5):
        s.check(*s.run(), want=want)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim,drafts", [(128, 9), (128, 16), (64, 17)])
def test_many_short_sequences(torch, dim, drafts, dtype):
    """Sequences enough to fill the GPU with few keys each: none, one, part of a tile, a tile and one more."""
    rng = np.random.default_rng(drafts)
    ctx = [0, 1, 63, 64, 65, 128, 200] + [int(v) for v in rng.integers(0, 150, 33)]
    count = [drafts, 1, 0, drafts] + [int(v) for v in rng.integers(0, drafts + 1, 36)]
    _go(torch, ctx, count, 16, 4, dim, 16, dtype=dtype, seed=drafts)


@pytest.mark.parametrize("ctx", [470, 503, 600, 2100])
@pytest.mark.parametrize("drafts", [9, 15, 16])
def test_rows_of_half_a_group(torch, ctx, drafts):
    """33 to 64 rows a kv head, one sequence and a few."""
    _go(torch, [ctx], [drafts], 8, 2, 128, 32, seed=ctx)
    _go(torch, [ctx, 3, 900], [drafts, 9, 2], 4, 1, 128, 48, seed=ctx)
