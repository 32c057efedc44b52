"""Cases of what a verify step does behind its logits and with its cache:
probabilities of the kept tokens, verification of drafted trees against the
target's and the drafter's probabilities, the accepted drafts' move to the end of
the context, pages of the cache turned into 8 bits, and tree attention over a
cache whose older pages are in 8 bits.  `run` computes them in their plain form,
or through the library's entry points where `own` is true; `exact` computes the
definitions in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
VOCAB = 129280


def listed():
    return [
        # the five rows of one verify step, every filter at once: latency
        dict(name="probs_verify_5", op="probs", dtype="f32", rows=5, vocab=VOCAB, mix="all"),
        # a server's batch, a different setting in each row
        dict(name="probs_batch_256", op="probs", dtype="f32", rows=256, vocab=VOCAB, mix="mixed"),
        # a chain of four drafts behind the last token of one conversation: latency
        dict(name="verify_chain_5", op="verify", seqs=1, tokens=5, side=0, ragged=False, vocab=VOCAB, draft="probs"),
        # a server's batch of small trees
        dict(name="verify_trees_64", op="verify", seqs=64, tokens=12, side=3, ragged=True, vocab=VOCAB, draft="probs"),
        # one conversation's accepted drafts, all layers: latency
        dict(name="commit_tree_1", op="commit", dtype="bf16", seqs=1, tokens=16, layers=32, kv=8, dim=128, page=64, ctx=8191),
        # a server's batch of large trees, heads of 64, pages that are no power of two
        dict(name="commit_batch_64", op="commit", dtype="f16", seqs=64, tokens=63, layers=32, kv=5, dim=64, page=48, ctx=500),
        # a page that one conversation has filled, in each of the layers
        dict(name="quantize_page_1", op="quantize", dtype="bf16", pages=1, layers=32, kv=8, dim=128, page=64, block=64),
        # a long prompt's pages, a scale for each 16 tokens
        dict(name="quantize_prompt_341", op="quantize", dtype="f16", pages=341, layers=4, kv=8, dim=128, page=48, block=16),
        # one token of one short conversation: latency
        dict(name="attn8_decode_300", op="attn8", dtype="bf16", seqs=1, tokens=1, ragged=False, heads=32, kv=8, dim=128,
             ctx=300, page=16, block=16),
        # a server's batch: ragged lengths and trees, heads of 64, pages that are no power of two
        dict(name="attn8_ragged_24", op="attn8", dtype="f16", seqs=24, tokens=13, ragged=True, heads=30, kv=5, dim=64,
             ctx=30000, page=48, block=16),
        # a large tree for several conversations: most arithmetic
        dict(name="attn8_tree64_8", op="attn8", dtype="bf16", seqs=8, tokens=64, ragged=False, heads=64, kv=8, dim=128,
             ctx=16000, page=32, block=32),
        # two long documents, decode plus three drafts: most bytes
        dict(name="attn8_long_131000", op="attn8", dtype="bf16", seqs=2, tokens=4, ragged=False, heads=32, kv=8, dim=128,
             ctx=131000, page=128, block=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.7e15)


def draw(rng):
    op = rng.choice(["probs", "verify", "commit", "quantize", "attn8", "attn8"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "probs":
            c = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), rows=_log(rng, 1, 256), vocab=_log(rng, 1000, VOCAB),
                     mix=rng.choice(["plain", "nucleus", "all", "mixed"]))
        elif op == "verify":
            c = dict(op=op, seqs=_log(rng, 1, 64), tokens=_log(rng, 1, 64), side=rng.choice([0, 0, 1, 2, 3]),
                     ragged=rng.random() < 0.6, vocab=_log(rng, 1000, VOCAB), draft=rng.choice(["probs", "probs", "point"]))
            if c["seqs"] * c["tokens"] > 64 * 12:  # (the rows of both distributions fit in 0.8 GB)
                continue
        elif op == "commit":
            c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), seqs=_log(rng, 1, 64), tokens=_log(rng, 6, 64),
                     layers=_log(rng, 1, 64), kv=rng.choice([1, 2, 5, 8]), dim=rng.choice([64, 96, 128, 256]),
                     page=rng.choice([16, 32, 48, 64, 128]), ctx=_log(rng, 1, 8191))
            if c["layers"] * c["kv"] * c["dim"] * (c["seqs"] * (c["tokens"] + 3 * c["page"])) > 400e6:
                continue
        elif op == "quantize":
            page = rng.choice([16, 32, 48, 64, 128])
            c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), pages=_log(rng, 1, 341), layers=_log(rng, 1, 64),
                     kv=rng.choice([1, 2, 5, 8]), dim=rng.choice([64, 96, 128, 256]), page=page, block=rng.choice([16, page]))
        else:
            kv, group, page = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 4, 6, 7, 8, 16]), rng.choice([16, 32, 48, 64, 128])
            c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), seqs=_log(rng, 1, 64), tokens=_log(rng, 1, 64),
                     ragged=rng.random() < 0.6, heads=kv * group, kv=kv, dim=rng.choice([64, 128, 128, 256]),
                     ctx=_log(rng, 1, 131000), page=page, block=rng.choice([16, page]))
            if c["seqs"] * c["heads"] * c["tokens"] * c["ctx"] > 8 * 64 * 64 * 16000:
                continue
        if _cost(c) > most:
            continue
        return c


# -------------------------------------------------- shapes of the cases --

def _lengths(case):
    """(context, drafted tokens) of each sequence; the same for every seed, in another order."""
    rng = random.Random("%(seqs)d %(tokens)d %(ctx)d" % case)
    if not case["ragged"]:
        return [(case["ctx"], case["tokens"])] * case["seqs"]
    some = [(_log(rng, 1, case["ctx"]), rng.randint(1, case["tokens"])) for _ in range(case["seqs"])]
    some[-1] = (case["ctx"], case["tokens"])
    if len(some) > 2:
        some[0] = (0, some[0][1])  # a new conversation: drafts alone
    return some


def _old(case, ctx):
    """Places of a context that are in 8 bits: its full pages, but for the last of them where there are many."""
    full = ctx // case["page"]
    return (full - (full > 8)) * case["page"]


def _draft_counts(case):
    """Drafted tokens of each sequence (the last one has the most)."""
    rng = random.Random("%(seqs)d %(tokens)d" % case)
    if not case.get("ragged"):
        return [case["tokens"]] * case["seqs"]
    return [rng.randint(1, case["tokens"]) for _ in range(case["seqs"] - 1)] + [case["tokens"]]


def _drafted(n, side):
    """Parents of n drafts: the likeliest chain first, then (side > 0) that many others off each of its tokens, as long as
    there are some, and what is left as chains behind those."""
    main = n if not side else max(1, (n + side) // (side + 1))
    parents = list(range(-1, main - 1))
    for k in range(n - main):
        at = k // side if side else 0
        parents.append(at if at < main else main + k - main * side)
    return parents


def _moves(case):
    """The accepted drafts of each sequence: the beginning of the likeliest chain, then a side branch behind it."""
    rng = random.Random("%(seqs)d %(tokens)d" % case)
    some = []
    for _ in range(case["seqs"]):
        n = case["tokens"]
        main = max(1, n // 3)
        keep = rng.randint(1, max(1, main - 1))           # of the chain's tokens 0 .. main - 1
        most = min(main - keep, n - main)                 # no branch gets deeper than the chain
        first = rng.randint(main, n - most) if most else main
        some.append(list(range(keep)) + list(range(first, first + (rng.randint(1, most) if most else 0))))
    return some


def _tree_bits(rng, n):
    """Bits of the drafted tokens that each of n sees: itself and its ancestors."""
    rows = []
    for i in range(n):
        parent = rng.choice([i - 1, i - 1, rng.randrange(-1, i)]) if i else -1
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    return [r - (1 << 64) if r >> 63 else r for r in rows]


# ---------------------------------------------------------------- inputs --

def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _starts(counts):
    return _i32(np.cumsum([0] + counts).tolist())


def _logits(g, rows, vocab):
    """Logits as an output head gives them: a broad background and some forty likely tokens."""
    x = torch.randn((rows, vocab), generator=g, device="cuda") * 2.5
    likely = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")
    # the larger of two values where a place comes twice: a plain scatter would take either
    return x.scatter_reduce_(1, likely, torch.rand((rows, 40), generator=g, device="cuda") * 12 + 2, "amax")


def _to_8_bits(x, block):
    """x (pages, page, kv, dim) as e4m3 numbers and a scale for each `block` tokens and head: the least power of two that
    brings the largest magnitude to 448 or less (1 where all are zero)."""
    y = x.float().unflatten(1, (-1, block))                           # (pages, blocks, block, kv, dim)
    most = y.abs().amax(dim=(2, 4))
    m, e = torch.frexp(most)                                          # most = m 2^e, 1/2 <= m < 1; 448 = (7/8) 2^9
    e = torch.where(most > 0, (e - 9 + (m > 0.875)).clamp(-80, 120), torch.zeros_like(e))
    scale = (e + 127 << 23).int().view(torch.float32)                 # 2^e
    v = y / scale[:, :, None, :, None]
    return v.to(torch.float8_e4m3fn).flatten(1, 2), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, s = case["op"], {"case": case}

    def normal(*shape, dtype):
        if dtype == torch.float16:
            return torch.randn(shape, generator=g, device="cuda").to(dtype)
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def cache(*shape):
        """Keys or values: heads and channels of different magnitudes."""
        x = normal(*shape, dtype=DTYPES[case["dtype"]])
        return x.mul_(torch.exp2(torch.randint(-2, 3, shape[-2:], generator=g, device="cuda").float()).to(x.dtype))

    if op == "probs":
        n, mix = case["rows"], case["mix"]
        s["logits"] = _logits(g, n, case["vocab"]).to(DTYPES[case["dtype"]])
        kinds = [mix if mix != "mixed" else rng.choice(["plain", "nucleus", "top", "least", "all", "greedy"]) for _ in range(n)]
        pick = lambda f, off, *names: [f() if k in names else off for k in kinds]  # noqa: E731
        hot = [0.0 if k == "greedy" else rng.uniform(0.4, 1.4) for k in kinds]
        s["temperature"] = torch.tensor(hot, dtype=torch.float32).cuda()
        s["top_k"] = _i32(pick(lambda: _log(rng, 1, 1000), 0, "top", "all"))
        s["top_p"] = torch.tensor(pick(lambda: rng.uniform(0.5, 0.99), 1.0, "nucleus", "all"), dtype=torch.float32).cuda()
        s["min_p"] = torch.tensor(pick(lambda: rng.uniform(0.001, 0.1), 0.0, "least", "all"), dtype=torch.float32).cuda()
    elif op == "verify":
        counts = _draft_counts(case)
        rng.shuffle(counts)
        total, vocab = sum(counts), case["vocab"]
        x = _logits(g, total, vocab)
        s["probs"] = torch.softmax(x, 1)
        # the drafter's view of the same places: near the target's, and a little flatter
        q = torch.softmax(x.mul_(0.9).add_(torch.randn((total, vocab), generator=g, device="cuda"), alpha=0.7), 1)
        parents = [p for n in counts for p in _drafted(n, case["side"])]
        first = [a for a, n in zip(np.cumsum([0] + counts).tolist(), counts) for _ in range(n)]
        s["parent"], s["start"], s["max_tok"] = _i32(parents), _starts(counts), max(counts)
        at = torch.tensor([f + max(p, 0) for f, p in zip(first, parents)]).cuda()
        # each draft drawn from the drafter's distribution at its parent
        u = torch.rand((total, 1), generator=g, device="cuda", dtype=torch.float64)
        drawn = torch.cat([torch.searchsorted(torch.cumsum(q[i].double(), 1), v) for i, v in zip(at.split(64), u.split(64))])
        s["tokens"] = drawn[:, 0].clamp_max(vocab - 1).int()
        s["draft"] = q if case["draft"] == "probs" else None
        s["u"] = torch.rand(total, generator=g, device="cuda")
        s["u_next"] = torch.rand(case["seqs"], generator=g, device="cuda")
    elif op == "commit":
        page, moves = case["page"], _moves(case)
        rng.shuffle(moves)
        n, width = case["seqs"], -(-(case["ctx"] + case["tokens"]) // page)
        tail = min(width, 1 + -(-case["tokens"] // page))  # pages of a sequence that the drafts can touch, and the one before
        # the older pages, which a commit does not touch, are one page that all sequences' tables name
        s["kc"], s["vc"] = (cache(case["layers"], n * tail + 1, page, case["kv"], case["dim"]) for _ in "kv")
        ids = torch.randperm(n * tail, generator=g, device="cuda").to(torch.int32).view(n, tail)
        s["table"] = torch.full((n, width), n * tail, dtype=torch.int32, device="cuda")
        s["table"][:, width - tail:] = ids
        s["ctx"] = torch.full((n,), case["ctx"], dtype=torch.int32, device="cuda")
        s["path"] = _i32([m + [-1] * (case["tokens"] - len(m)) for m in moves])
        s["count"] = _i32([len(m) for m in moves])
    elif op == "quantize":
        n, more = case["pages"], case["pages"] + 2
        shape = (case["layers"], more, case["page"], case["kv"], case["dim"])
        s["kc"], s["vc"] = (cache(*shape) for _ in "kv")
        s["k8"], s["v8"] = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
        s["ks"], s["vs"] = (torch.ones((case["layers"], more, case["page"] // case["block"], case["kv"]), device="cuda") for _ in "kv")
        s["src"], s["dst"] = (torch.randperm(more, generator=g, device="cuda")[:n].int() for _ in "sd")
    else:
        some = _lengths(case)
        rng.shuffle(some)
        page, old = case["page"], [_old(case, c) for c, _ in some]
        need8, need = [o // page for o in old], [-(-(c + n) // page) - o // page for (c, n), o in zip(some, old)]
        total = sum(n for _, n in some)
        s["q"] = normal(total, case["heads"], case["dim"], dtype=DTYPES[case["dtype"]])
        pages8 = sum(need8) + 2
        for x, y in (("k8", "ks"), ("v8", "vs")):
            s[x], s[y] = _to_8_bits(cache(pages8, page, case["kv"], case["dim"]), case["block"])
        s["kc"], s["vc"] = (cache(sum(need) + 2, page, case["kv"], case["dim"]) for _ in "kv")
        s["table8"], s["table"] = (torch.full((len(some), w), -1, dtype=torch.int32) for w in
                                   (max(1, max(need8)), max(-(-(c + n) // page) for c, n in some)))
        ids8, ids = (torch.randperm(k, generator=g, device="cuda").to(torch.int32).cpu() for k in (pages8, sum(need) + 2))
        a = b = 0
        for i, (w8, w) in enumerate(zip(need8, need)):
            s["table8"][i, :w8] = ids8[a:a + w8]
            s["table"][i, w8:w8 + w] = ids[b:b + w]  # the pages that went to 8 bits are no longer there
            a, b = a + w8, b + w
        s["table8"], s["table"] = s["table8"].cuda(), s["table"].cuda()
        s["old"], s["ctx"], s["start"] = _i32(old), _i32([c for c, _ in some]), _starts([n for _, n in some])
        s["mask"] = torch.tensor([b for _, n in some for b in _tree_bits(rng, n)], dtype=torch.int64).cuda()
        s["max_tok"], s["max_old"] = max(n for _, n in some), max(old)
        s["max_new"] = max(c + n - o for (c, n), o in zip(some, old))
    return s


# ----------------------------------------------------------- plain forms --

def _plain_probs(s):
    x = s["logits"].double()
    n, vocab = x.shape
    greedy = (s["temperature"] == 0)[:, None]
    t = torch.where(greedy, torch.ones_like(x[:, :1]), s["temperature"].double()[:, None])
    sx, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((sx - sx[:, :1]) / t)
    rank = torch.arange(vocab, device=x.device)[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), vocab)[:, None]
    w = w * (rank < k)
    before = torch.cumsum(w, 1) - w
    keep = (before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True)) | (s["top_p"] >= 1)[:, None]
    keep &= (w >= s["min_p"].double()[:, None]) | (rank == 0)
    w = torch.where(greedy, (rank == 0).double(), w * keep)
    return torch.zeros_like(w).scatter_(1, order, w / w.sum(1, keepdim=True)).float()


def _plain_verify(s):
    p, q, first = s["probs"], s["draft"], s["start"][:-1].long()
    n, (total, vocab), most = first.numel(), p.shape, s["max_tok"]
    dev, count = p.device, (s["start"][1:] - s["start"][:-1]).long()
    seq = torch.arange(n, device=dev)
    at = torch.zeros(n, dtype=torch.long, device=dev)  # the last accepted draft
    path = torch.full((n, most), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    taken = torch.ones(n, dtype=torch.int32, device=dev)
    rest, left = p[first].double(), torch.ones(n, dtype=torch.float64, device=dev)  # what may still be drawn at it, and its mass
    for i in range(1, most):  # children come behind their parents, so one look at each draft is enough
        row = (first + i).clamp_max(total - 1)
        asked = (i < count) & (s["parent"][row].long() == at)
        x = s["tokens"][row].long()
        here = q[first + at].double() if q is not None else torch.zeros_like(rest).scatter_(1, x[:, None], 1.0)
        taking = asked & (s["u"][row].double() * here[seq, x] * left < rest[seq, x])
        path[seq, taken.long().clamp_max(most - 1)] = torch.where(taking, i, path[seq, taken.long().clamp_max(most - 1)])
        taken += taking.int()
        at = torch.where(taking, i, at)
        less = (rest - left[:, None] * here).clamp_min(0)
        if q is None:
            less = rest * (here == 0)
        less_left = less.sum(1) if q is not None else left - rest[seq, x]
        refused = asked & ~taking
        rest = torch.where(taking[:, None], p[row].double(), torch.where(refused[:, None], less, rest))
        left = torch.where(taking, torch.ones_like(left), torch.where(refused, less_left, left))
    sums = torch.cumsum(rest, 1)
    after = (sums <= s["u_next"].double()[:, None] * sums[:, -1:]).sum(1).clamp_max(vocab - 1)
    return {"path": path, "count": taken, "next": after.int()}


def _plain_commit(s):
    page, kc, vc = s["case"]["page"], s["kc"].flatten(1, 2), s["vc"].flatten(1, 2)
    n, most = s["path"].shape
    there = torch.arange(most, device=kc.device)[None, :] < s["count"][:, None]
    to = s["ctx"].long()[:, None] + torch.arange(most, device=kc.device)
    by = s["ctx"].long()[:, None] + s["path"].long()
    slot = lambda x: (s["table"].long().gather(1, x // page) * page + x % page)[there]  # noqa: E731
    a, b = slot(torch.where(there, by, 0)), slot(torch.where(there, to, 0))
    kc[:, b], vc[:, b] = kc[:, a], vc[:, a]
    return {"kc": s["kc"], "vc": s["vc"], "ctx": s["ctx"] + s["count"]}


def _plain_quantize(s):
    c = s["case"]
    for x, x8, xs in ((s["kc"], s["k8"], s["ks"]), (s["vc"], s["v8"], s["vs"])):
        v, scale = _to_8_bits(x[:, s["src"].long()].flatten(0, 1), c["block"])
        x8.view(torch.uint8)[:, s["dst"].long()] = v.view(torch.uint8).unflatten(0, (c["layers"], -1))
        xs[:, s["dst"].long()] = scale.unflatten(0, (c["layers"], -1))
    return {"k8": s["k8"], "v8": s["v8"], "ks": s["ks"], "vs": s["vs"]}


def _plain_attention(s):
    q, c = s["q"], s["case"]
    total, heads, dim = q.shape
    page, kv, block = c["page"], c["kv"], c["block"]
    n, most, length, group = s["ctx"].numel(), s["max_tok"], int(s["table"].shape[1]) * page, heads // kv
    tok = torch.arange(total, device=q.device)
    seq = torch.searchsorted(s["start"][1:].long(), tok, right=True)
    at = tok - s["start"].long()[seq]
    where = torch.arange(length, device=q.device)
    place = s["table"].long().clamp_min(0)[:, where // page] * page + where % page               # (n, length)
    where8 = where[:s["table8"].shape[1] * page]
    place8 = s["table8"].long().clamp_min(0)[:, where8 // page] * page + where8 % page
    is8 = (where8[None, :] < s["old"][:, None])[:, :, None, None]

    def whole(recent, x8, scale):
        """The sequences' keys or values in fp32 (n, length, kv, dim)."""
        x = recent.flatten(0, 1)[place].float()
        y = x8.view(torch.uint8).flatten(0, 1)[place8].view(torch.float8_e4m3fn).float()
        y *= scale.repeat_interleave(block, 1).flatten(0, 1)[place8][..., None]
        m = min(length, where8.numel())
        x[:, :m] = torch.where(is8[:, :m], y[:, :m], x[:, :m])
        return x

    k = whole(s["kc"], s["k8"], s["ks"])
    pad = q.new_zeros((n, most, heads, dim), dtype=torch.float32)
    pad[seq, at] = q.float()
    qs = pad.view(n, most, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, most * group, dim)
    score = qs @ k.permute(0, 2, 3, 1) * dim ** -0.5                          # (n, kv, most*group, length)
    del k
    bits = torch.zeros((n, most), dtype=torch.int64, device=q.device)
    bits[seq, at] = s["mask"]
    draft = where[None, :] - s["ctx"].long()[:, None]                         # (n, length)
    count = (s["start"][1:] - s["start"][:-1]).long()
    seen = (bits[:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    seen = (draft < 0)[:, None, :] | ((draft >= 0) & (draft < count[:, None]))[:, None, :] & (seen == 1)
    score = score.masked_fill(~seen[:, None, :, None, :].expand(n, 1, most, group, length).reshape(n, 1, most * group, length), -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(score - top)
    z = e.sum(-1, keepdim=True)
    v = whole(s["vc"], s["v8"], s["vs"])
    o = torch.where(z > 0, (e @ v.permute(0, 2, 1, 3)) / z, torch.zeros_like(z))
    lse = torch.where(z > 0, top + torch.log(z), torch.full_like(z, -math.inf))
    o, lse = (x.view(n, kv, most, group, -1).permute(0, 2, 1, 3, 4).reshape(n, most, heads, -1)[seq, at] for x in (o, lse))
    return {"out": o.to(q.dtype), "lse": lse[..., 0]}


def run(s):
    op = s["case"]["op"]
    if own:
        from verify_matvec_gb300 import cbq
        if op == "probs":
            return cbq.cbq_probs(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        if op == "verify":
            path, count, after = cbq.cbq_verify(s["probs"], s["draft"], s["tokens"], s["parent"], s["start"], s["u"], s["u_next"],
                                                max_tok=s["max_tok"])
            return {"path": path, "count": count, "next": after}
        if op == "commit":
            ctx = cbq.cbq_kv_commit(s["kc"], s["vc"], s["table"], s["ctx"], s["path"], s["count"])
            return {"kc": s["kc"], "vc": s["vc"], "ctx": ctx}
        if op == "quantize":
            cbq.cbq_kv_quantize(s["kc"], s["vc"], s["src"], s["k8"], s["v8"], s["ks"], s["vs"], s["dst"])
            return {"k8": s["k8"], "v8": s["v8"], "ks": s["ks"], "vs": s["vs"]}
        out, lse = cbq.cbq_tree_attention8(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["table8"], s["old"], s["kc"], s["vc"],
                                           s["table"], s["ctx"], s["start"], s["mask"], max_tok=s["max_tok"],
                                           max_old=s["max_old"], max_new=s["max_new"], with_lse=True)
        return {"out": out, "lse": lse}
    return {"probs": _plain_probs, "verify": _plain_verify, "commit": _plain_commit, "quantize": _plain_quantize,
            "attn8": _plain_attention}[op](s)


def work(case):
    op = case["op"]
    if op == "probs":  # the logits once, the probabilities once
        return {"bytes": case["rows"] * (case["vocab"] * (SIZE[case["dtype"]] + 4) + 16), "flops": 4 * case["rows"] * case["vocab"]}
    if op == "verify":  # of each sequence, the row (or the two) of the place where it draws
        rows = 1 + (case["draft"] == "probs")
        return {"bytes": case["seqs"] * (rows * case["vocab"] * 4 + 12) + sum(_draft_counts(case)) * 24,
                "flops": 3 * case["seqs"] * case["vocab"]}
    if op == "commit":  # what moves, read and written
        moved = sum(a != b for m in _moves(case) for a, b in enumerate(m))
        return {"bytes": 4 * moved * case["layers"] * case["kv"] * case["dim"] * SIZE[case["dtype"]] + 4 * case["seqs"] * (case["tokens"] + 3),
                "flops": 0}
    if op == "quantize":
        values = 2 * case["pages"] * case["layers"] * case["page"] * case["kv"] * case["dim"]
        return {"bytes": values * (SIZE[case["dtype"]] + 1) + 4 * values // (case["block"] * case["dim"]) + 8 * case["pages"],
                "flops": 2 * values}
    d, some = SIZE[case["dtype"]], _lengths(case)
    old, toks = sum(_old(case, c) for c, _ in some), sum(n for _, n in some)
    recent = sum(c + n for c, n in some) - old
    return {"bytes": 2 * case["kv"] * (old * case["dim"] + 4 * old // case["block"] + recent * case["dim"] * d)
            + toks * case["heads"] * (2 * case["dim"] * d + 4),
            "flops": 4 * sum((c + n) * n for c, n in some) * case["heads"] * case["dim"]}


# ------------------------------------------------- definitions in 64 bits --

def _exact_probs(s):
    out = []
    for i, row in enumerate(s["logits"].double().cpu().numpy()):
        t, k, p, m = (float(s[x][i]) for x in ("temperature", "top_k", "top_p", "min_p"))
        order = np.lexsort((np.arange(row.size), -row))
        probs = np.zeros(row.size)
        if t == 0:
            probs[order[0]] = 1.0
        else:
            order = order[:int(k)] if k else order
            w = np.exp((row[order] - row[order[0]]) / t)
            sums = np.cumsum(w)
            kept = order.size if p >= 1 else int(np.searchsorted(sums, p * sums[-1])) + 1
            kept = max(1, min(kept, int(np.sum(w >= m))))
            probs[order[:kept]] = w[:kept] / w[:kept].sum()
        out.append(probs)
    return np.stack(out)


def _exact_verify(s):
    start, parent, tokens, u, after = (s[x].tolist() for x in ("start", "parent", "tokens", "u", "u_next"))
    path = np.full((len(after), s["max_tok"]), -1, np.int32)
    count, chosen = np.zeros(len(after), np.int32), np.zeros(len(after), np.int32)
    for i, (a, b) in enumerate(zip(start, start[1:])):
        at = 0
        while True:
            path[i, count[i]] = at
            count[i] += 1
            rest = s["probs"][a + at].double().cpu().numpy()
            q = None if s["draft"] is None else s["draft"][a + at].double().cpu().numpy()
            mass, into = 1.0, None
            for j in range(at + 1, b - a):
                if parent[a + j] != at:
                    continue
                x = tokens[a + j]
                if u[a + j] * mass * (1.0 if q is None else q[x]) < rest[x]:
                    into = j
                    break
                if q is None:
                    mass -= rest[x]
                    rest[x] = 0
                else:
                    rest = np.maximum(rest - mass * q, 0)
                    mass = rest.sum()
            if into is None:
                break
            at = into
        sums = np.cumsum(rest)
        chosen[i] = min(int(np.searchsorted(sums, after[i] * sums[-1], side="right")), rest.size - 1)
    return {"path": path, "count": count, "next": chosen}


def _exact_commit(s):
    page, table = s["case"]["page"], s["table"].tolist()
    kc, vc = s["kc"].clone(), s["vc"].clone()
    for i, (c, n, path) in enumerate(zip(s["ctx"].tolist(), s["count"].tolist(), s["path"].tolist())):
        for a, b in enumerate(path[:n]):
            (pa, ta), (pb, tb) = divmod(c + b, page), divmod(c + a, page)
            for x in (kc, vc):
                x[:, table[i][pb], tb] = x[:, table[i][pa], ta].clone()
    return {"kc": kc.double(), "vc": vc.double(), "ctx": (s["ctx"] + s["count"]).cpu().numpy()}


def _exact_quantize(s):
    """Rounding to three bits behind the leading one (down to 2^-9), halves to even, by division and rounding."""
    c, out = s["case"], {}
    src, dst = s["src"].long(), s["dst"].long()
    for x, to, name, names in (("kc", "k8", "k8", "ks"), ("vc", "v8", "v8", "vs")):
        v8, scales = s[to].double(), s[names].double()
        y = s[x][:, src].double().unflatten(2, (-1, c["block"]))
        most = y.abs().amax((3, 5))
        e = torch.ceil(torch.log2(most.clamp_min(1e-300) / 448))
        e = e + (448 * torch.exp2(e) < most) - (448 * torch.exp2(e - 1) >= most).double()
        scale = torch.where(most > 0, torch.exp2(e.clamp(-80, 120)), torch.ones_like(e))
        y = y / scale[:, :, :, None, :, None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        v8[:, dst] = (torch.round(y / step) * step).flatten(2, 3)
        scales[:, dst] = scale
        out[name], out[names] = v8, scales
    return {k: out[k] for k in ("k8", "v8", "ks", "vs")}


def _exact_attention(s):
    case = s["case"]
    start, ctx, old, group = s["start"].tolist(), s["ctx"].tolist(), s["old"].tolist(), case["heads"] // case["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, c in enumerate(ctx):
        a, b, w8 = start[i], start[i + 1], old[i] // case["page"]
        pages8, pages = s["table8"][i, :w8].long(), s["table"][i, w8:-(-(c + b - a) // case["page"])].long()
        allow = torch.ones(b - a, c + b - a, dtype=torch.bool, device="cuda")
        for j, m in enumerate(s["mask"][a:b].tolist()):
            allow[j, c:] = torch.tensor([bool(m >> x & 1) for x in range(b - a)], device="cuda")
        for g in range(case["kv"]):
            both = []
            for recent, x8, scale in ((s["kc"], s["k8"], s["ks"]), (s["vc"], s["v8"], s["vs"])):
                y = x8[:, :, g].view(torch.uint8)[pages8].view(torch.float8_e4m3fn).double()
                y = y * scale[pages8][:, :, g].double().repeat_interleave(case["block"], 1)[..., None]
                both.append(torch.cat([y.flatten(0, 1), recent[:, :, g][pages].double().flatten(0, 1)])[:c + b - a])
            k, v = both
            for h in range(g * group, (g + 1) * group):
                e = (s["q"][a:b, h].double() @ k.T / math.sqrt(case["dim"])).masked_fill(~allow, -math.inf)
                lse[a:b, h] = torch.logsumexp(e, 1)
                out[a:b, h] = torch.exp(e - lse[a:b, h, None]) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "attn8" and work(case)["flops"] > 5e12:
        return None
    return {"probs": _exact_probs, "verify": _exact_verify, "commit": _exact_commit, "quantize": _exact_quantize,
            "attn8": _exact_attention}[case["op"]](prepare(case, seed))
