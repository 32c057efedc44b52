"""The calls behind the logits as they are used together: several verify rounds
of a few conversations over a paged cache of two layers.  In each round the
drafts' keys and values are appended, the trees verified against the target's and
the drafter's distributions, the accepted ones moved behind their contexts, pages
that are full put into 8 bits, and the tree attention reads both kinds.  A
plain account of every place is kept beside it and compared after each step."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("dtype,heads,kv,dim,page,block", [("bfloat16", 8, 2, 128, 16, 16), ("float16", 20, 1, 64, 8, 4)])
def test_rounds(torch, dtype, heads, kv, dim, page, block):
    rng = np.random.default_rng(5)
    g = torch.Generator(device="cuda").manual_seed(5)
    dt, layers, n_seq, most, V, width = getattr(torch, dtype), 2, 3, 9, 700, 24
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    pages = n_seq * width
    kc, vc = (torch.zeros((layers, pages, page, kv, dim), dtype=dt, device="cuda") for _ in "kv")
    k8, v8 = (torch.zeros((layers, pages, page, kv, dim), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros((layers, pages, page // block, kv), device="cuda") for _ in "kv")
    table, table8 = (rng.permutation(pages).reshape(n_seq, width) for _ in range(2))
    ctx, old = np.array([0, 37, 5], np.int32), np.zeros(n_seq, np.int32)
    account = [[[], []] for _ in range(n_seq)]  # of each place, what its key and value stand for (layers, kv, dim)
    for s in range(n_seq):
        for p in range(ctx[s]):
            for x, cache in enumerate((kc, vc)):
                value = torch.randn((layers, kv, dim), generator=g, device="cuda").to(dt)
                cache[:, table[s][p // page], p % page] = value
                account[s][x].append(num(value))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    turns = cbq.cbq_rope_turns(dim)
    for _ in range(6):
        sizes = rng.integers(1, most + 1, n_seq)
        start = np.cumsum([0] + list(sizes))
        total = int(start[-1])
        parent = np.concatenate([[-1] + [int(rng.integers(0, i)) for i in range(1, n)] for n in sizes])
        bits = np.zeros(total, np.int64)
        for s in range(n_seq):
            for i in range(sizes[s]):
                r = start[s] + i
                bits[r] = (bits[start[s] + parent[r]] if i else 0) | 1 << i
        # the drafts' keys and values, behind their contexts (position 0 for all: nothing turns)
        place = np.concatenate([ctx[s] + np.arange(sizes[s]) for s in range(n_seq)])
        of = np.repeat(np.arange(n_seq), sizes)
        slots = torch.from_numpy(table[of, place // page] * page + place % page).cuda()
        new = [[torch.randn((total, kv, dim), generator=g, device="cuda").to(dt) for _ in range(layers)] for _ in "kv"]
        q = torch.randn((total, heads, dim), generator=g, device="cuda").to(dt)
        for layer in range(layers):
            cbq.cbq_rope_append(q, new[0][layer], new[1][layer], i32(np.zeros(total)), slots, turns, kc[layer], vc[layer], err=err)
        # attention of the drafts in each layer, over what is old and what is recent
        lim = dict(max_tok=int(sizes.max()), max_old=int(old.max()), max_new=int((ctx + sizes - old).max()))
        for layer in range(layers):
            out, lse = cbq.cbq_tree_attention8(q, k8[layer], v8[layer], ks[layer], vs[layer], i32(table8), i32(old), kc[layer], vc[layer],
                                               i32(table), i32(ctx), i32(start), torch.from_numpy(bits).cuda(), **lim,
                                               with_lse=True, err=err, out=torch.empty(q.shape, device="cuda"))
            seqs = []
            for s in range(n_seq):
                k, v = (np.concatenate([np.array([a[layer] for a in account[s][x]]).reshape(-1, kv, dim),
                                        num(new[x][layer][start[s]:start[s + 1]])]) for x in range(2))
                seen = np.array([[p < ctx[s] or bool(int(bits[start[s] + i]) >> int(p - ctx[s]) & 1) for p in range(len(k))] for i in range(sizes[s])])
                seqs.append((start[s], k, v, seen))
            want, want_lse, absv, big = behind_ref.attention(num(q), seqs, dim ** -0.5)
            # scores and weights as in tests/test_gpu_tree_attention8.py, results in fp32
            delta = (dim + 8) * 2.0 ** -24 * big
            lim_out = absv * (torch.finfo(dt).eps / 2 + 4 * delta[..., None] + 300 * 2.0 ** -24) + 300 * 2.0 ** -25 * 8
            assert np.all(np.abs(num(out) - want) <= lim_out)
            assert np.all(np.abs(num(lse) - want_lse) <= delta + 2.0 ** -22 + 2.0 ** -23 * (np.abs(want_lse) + 24) + 300 * 2.0 ** -24)
        # the trees against the target's and the drafter's distributions of the same logits' neighbours
        x = torch.randn((total, V), generator=g, device="cuda") * 2
        hot, top = torch.full((total,), 0.8, device="cuda"), torch.full((total,), 0.97, device="cuda")
        p = cbq.cbq_probs(x, hot, None, top, None)
        d = cbq.cbq_probs(x + torch.randn((total, V), generator=g, device="cuda") * 0.5, hot, None, None, None)
        rows = num(d)
        tokens = np.array([0 if parent[r] < 0 else rng.choice(V, p=rows[start[of[r]] + parent[r]] / rows[start[of[r]] + parent[r]].sum())
                           for r in range(total)])
        u, un = rng.random(total, dtype=np.float32), rng.random(n_seq, dtype=np.float32)
        path, count, after = cbq.cbq_verify(p, d, i32(tokens), i32(parent), i32(start), torch.from_numpy(u).cuda(),
                                            torch.from_numpy(un).cuda(), max_tok=most, err=err)
        for s in range(n_seq):
            a, b = start[s], start[s + 1]
            want, token, margin = behind_ref.verify(num(p)[a:b], rows[a:b], tokens[a:b], parent[a:b], u[a:b], un[s])
            assert margin < 2.0 ** -40 or (path[s].tolist()[:len(want)] == want and int(count[s]) == len(want) and int(after[s]) == token)
        # the accepted ones move; the account gets the same
        ctx_dev = cbq.cbq_kv_commit(kc, vc, i32(table), i32(ctx), path, count, err=err)
        for s in range(n_seq):
            for i in path[s].tolist()[:int(count[s])]:
                for y in range(2):
                    account[s][y].append(np.stack([num(new[y][layer][start[s] + i]) for layer in range(layers)]))
        ctx = ctx_dev.cpu().numpy()
        assert list(ctx) == [len(a[0]) for a in account]
        # full pages into 8 bits, and the account with them; then nothing reads them in 16
        src, dst = [], []
        for s in range(n_seq):
            while ctx[s] - old[s] >= page:
                src.append(table[s][old[s] // page])
                dst.append(table8[s][old[s] // page])
                for y in range(2):
                    there = np.stack(account[s][y][old[s]:old[s] + page], 1)  # (layers, page, kv, dim)
                    v, scale = behind_ref.quantize(there, block)
                    stand = v * np.repeat(scale, block, 1)[..., None]
                    for t in range(page):
                        account[s][y][old[s] + t] = stand[:, t]
                old[s] += page
        if src:
            cbq.cbq_kv_quantize(kc, vc, i32(src), k8, v8, ks, vs, i32(dst), err=err)
            kc[:, src], vc[:, src] = float("nan"), float("nan")
        assert int(err) == 0
    assert old.max() >= 2 * page
