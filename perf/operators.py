"""Cases of the operators around the quantized products of a verify step: rotary
positions (of a tensor, and of new tokens on their way into a paged cache),
attention of a tree of drafted tokens over that cache, and sampling from the
logits.  `run` computes them in their plain form, or through the library's entry
points where `own` is true; `exact` computes the definitions in 64 bits."""
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
        # a prefill chunk's queries, half layout, whole heads
        dict(name="rope_prefill_8192", op="rope", dtype="bf16", tokens=8192, heads=32, dim=128, rot=128, off=0,
             layout="half", scaling="none", far=1 << 17),
        # a few tokens, neighbours paired, the last 64 of 192 values of a head, frequencies stretched for a long context
        dict(name="rope_part_37", op="rope", dtype="f32", tokens=37, heads=16, dim=192, rot=64, off=128,
             layout="pairs", scaling="turns", far=1 << 20),
        # one decode step plus four drafts: fp32 products into a bf16 cache
        dict(name="append_verify_5", op="append", dtype="f32", cache="bf16", tokens=5, heads=32, kv=8, dim=128, rot=128,
             off=0, layout="half", scaling="none", far=1 << 17, page=64, pages=256),
        # a prompt's chunk written to the cache, part of the head rotated
        dict(name="append_prompt_4095", op="append", dtype="bf16", cache="bf16", tokens=4095, heads=32, kv=8, dim=128,
             rot=64, off=64, layout="pairs", scaling="index", far=1 << 17, page=16, pages=512),
        # one token of one short conversation: latency
        dict(name="attn_decode_300", op="attn", dtype="bf16", seqs=1, tokens=1, ragged=False, heads=32, kv=8, dim=128,
             ctx=300, page=16),
        # decode plus four drafts of one conversation (the widest verify of the matvec)
        dict(name="attn_verify5_8191", op="attn", dtype="bf16", seqs=1, tokens=5, ragged=False, heads=32, kv=8, dim=128,
             ctx=8191, page=64),
        # a server's batch: ragged lengths and trees, heads of 64, pages that are no power of two
        dict(name="attn_ragged_24", op="attn", dtype="f16", seqs=24, tokens=13, ragged=True, heads=30, kv=5, dim=64,
             ctx=30000, page=48),
        # a large tree for several conversations: most arithmetic
        dict(name="attn_tree64_8", op="attn", dtype="bf16", seqs=8, tokens=64, ragged=False, heads=64, kv=8, dim=128,
             ctx=16000, page=32),
        # two long documents, decode plus three drafts: most bytes
        dict(name="attn_long_131000", op="attn", dtype="bf16", seqs=2, tokens=4, ragged=False, heads=32, kv=8, dim=128,
             ctx=131000, page=128),
        # one row of the output head's logits
        dict(name="sample_1", op="sample", dtype="f32", rows=1, vocab=VOCAB, mix="nucleus"),
        # the five rows of a verify step, every filter at once
        dict(name="sample_verify_5", op="sample", dtype="f32", rows=5, vocab=VOCAB, mix="all"),
        # a server's batch, a different setting in each row
        dict(name="sample_batch_256", op="sample", dtype="f32", rows=256, vocab=VOCAB, mix="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.8e15)


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "sample"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op in ("rope", "append"):
            dim = rng.choice([64, 96, 128, 192, 256])
            rot = rng.choice([dim, dim // 2, 64, 32])
            c = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), tokens=_log(rng, 1, 8192),
                     heads=rng.choice([1, 5, 8, 16, 30, 32, 64]), dim=dim, rot=rot, off=rng.choice([0, dim - rot]),
                     layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["none", "linear", "turns", "index"]),
                     far=1 << rng.randrange(12, 21))
            if op == "append":
                page = rng.choice([1, 16, 32, 48, 64, 128])
                c.update(cache=rng.choice(["bf16", "f16"]), kv=rng.choice([1, 2, 5, 8]), page=page)
                c["pages"] = -(-2 * c["tokens"] // page) + 3
                if c["dtype"] != "f32":
                    c["cache"] = c["dtype"]
        elif op == "attn":
            kv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 4, 6, 7, 8, 16])
            c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), seqs=_log(rng, 1, 64), tokens=_log(rng, 1, 64),
                     ragged=rng.random() < 0.6, heads=kv * group, kv=kv, dim=rng.choice([64, 128, 128, 256]),
                     ctx=_log(rng, 1, 131000), page=rng.choice([16, 32, 48, 64, 128]))
            if c["seqs"] * c["heads"] * c["tokens"] * c["ctx"] > 8 * 64 * 64 * 16000:
                continue
        else:
            c = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), rows=_log(rng, 1, 256),
                     vocab=_log(rng, 1000, VOCAB), mix=rng.choice(["plain", "nucleus", "all", "mixed"]))
        if 3072 in c.values() or c.get("heads", 0) * c.get("dim", 0) == 3072 or _cost(c) > most:
            continue
        return c


# ---------------------------------------------------------------- inputs --

def _turns(case):
    """Turns a position (fp64, rot/2 of them): base 10000, stretched as the case says."""
    half, base, factor, length, low, high = case["rot"] // 2, 10000.0, 16.0, 8192.0, 1.0, 32.0
    t = np.array([base ** (-i / half) / (2 * math.pi) for i in range(half)])
    if case["scaling"] == "linear":
        return t / factor
    if case["scaling"] == "turns":  # kept where a context of `length` turns `high` times or more, divided where under `low`
        keep = np.clip((t * length - low) / (high - low), 0, 1)
        return t * keep + t / factor * (1 - keep)
    if case["scaling"] == "index":  # the same borders as places in the table, a straight line between them
        at = [half * math.log(length / (r * 2 * math.pi)) / math.log(base) for r in (high, low)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), half - 1)
        keep = 1 - np.clip((np.arange(half) - lo) / max(hi - lo, 1e-3), 0, 1)
        return t * keep + t / factor * (1 - keep)
    return t


def _magnitude(case):
    return 0.1 * math.log(16.0) + 1.0 if case["scaling"] in ("turns", "index") else 1.0


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


def _tree(rng, n):
    """Bits of the drafted tokens that each of n sees: itself and its ancestors."""
    rows = []
    for i in range(n):
        parent = rng.choice([i - 1, i - 1, rng.randrange(-1, i)]) if i else -1
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    return [r - (1 << 64) if r >> 63 else r for r in rows]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype if dtype != torch.float16 else torch.float32).to(dtype)

    s = {"case": case}
    if case["op"] in ("rope", "append"):
        n = case["tokens"]
        first = rng.randrange(max(1, case["far"] - n))
        s["pos"] = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
        s["turns"] = torch.from_numpy(_turns(case)).cuda()
        s["magnitude"] = _magnitude(case)
    if case["op"] == "rope":
        s["x"] = normal(n, case["heads"], case["dim"])
    elif case["op"] == "append":
        cdt = DTYPES[case["cache"]]
        s["q"], s["k"], s["v"] = normal(n, case["heads"], case["dim"]), normal(n, case["kv"], case["dim"]), normal(n, case["kv"], case["dim"])
        s["kc"], s["vc"] = (normal(case["pages"], case["page"], case["kv"], case["dim"], dtype=cdt) for _ in "kv")
        at = rng.randrange(case["page"])  # the sequence goes on inside a page
        pages = torch.randperm(case["pages"], generator=g, device="cuda")
        where = torch.arange(at, at + n, device="cuda")
        s["slots"] = pages[where // case["page"]] * case["page"] + where % case["page"]
    elif case["op"] == "attn":
        some = _lengths(case)
        rng.shuffle(some)
        page, need = case["page"], [-(-(c + n) // case["page"]) for c, n in some]
        total, width = sum(n for _, n in some), max(need)
        s["q"] = normal(total, case["heads"], case["dim"])
        s["kc"], s["vc"] = (normal(sum(need) + 2, page, case["kv"], case["dim"]) for _ in "kv")
        table = torch.zeros(len(some), width, dtype=torch.int32)
        ids, at = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32).cpu(), 0
        for i, w in enumerate(need):
            table[i, :w] = ids[at:at + w]
            at += w
        s["table"] = table.cuda()
        s["ctx"] = torch.tensor([c for c, _ in some], dtype=torch.int32).cuda()
        s["start"] = torch.tensor(np.cumsum([0] + [n for _, n in some]).tolist(), dtype=torch.int32).cuda()
        s["mask"] = torch.tensor([b for _, n in some for b in _tree(rng, n)], dtype=torch.int64).cuda()
        s["max_tok"], s["max_len"] = max(n for _, n in some), max(c + n for c, n in some)
    else:
        n, mix = case["rows"], case["mix"]
        x = torch.randn((n, case["vocab"]), generator=g, device="cuda") * 2.5
        likely = torch.randint(0, case["vocab"], (n, 40), generator=g, device="cuda")
        # the larger of two values where a place comes twice: a plain scatter would take either
        x.scatter_reduce_(1, likely, torch.rand((n, 40), generator=g, device="cuda") * 12 + 2, "amax")
        s["logits"] = x.to(dt)
        kinds = [mix if mix != "mixed" else rng.choice(["plain", "nucleus", "top", "least", "all", "greedy"]) for _ in range(n)]
        pick = lambda f, off, *names: [f() if k in names else off for k in kinds]  # noqa: E731
        hot = [0.0 if k == "greedy" else rng.uniform(0.4, 1.4) for k in kinds]
        s["temperature"] = torch.tensor(hot, dtype=torch.float32).cuda()
        s["top_k"] = torch.tensor(pick(lambda: _log(rng, 1, 1000), 0, "top", "all"), dtype=torch.int32).cuda()
        s["top_p"] = torch.tensor(pick(lambda: rng.uniform(0.5, 0.99), 1.0, "nucleus", "all"), dtype=torch.float32).cuda()
        s["min_p"] = torch.tensor(pick(lambda: rng.uniform(0.001, 0.1), 0.0, "least", "all"), dtype=torch.float32).cuda()
        s["u"] = torch.rand(n, generator=g, device="cuda")
    return s


# ----------------------------------------------------------- plain forms --

def _rotate(s, x):
    """x (tokens, heads, dim) in fp32 with the case's part of each head rotated; the angles in 64 bits."""
    c = s["case"]
    half, lo, hi = c["rot"] // 2, c["off"], c["off"] + c["rot"]
    t = s["pos"].double()[:, None] * s["turns"][None, :]
    a = 2 * math.pi * (t - torch.round(t))
    cos, sin = ((f(a) * s["magnitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    x = x.float()
    p = x[..., lo:hi]
    if c["layout"] == "half":
        a, b = p[..., :half], p[..., half:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = p[..., 0::2], p[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([x[..., :lo], r, x[..., hi:]], -1)


def _plain_attention(s):
    q, kc, vc = s["q"], s["kc"], s["vc"]
    total, heads, dim = q.shape
    page, kv = kc.shape[1], kc.shape[2]
    n, most, length, group = s["ctx"].numel(), s["max_tok"], s["max_len"], heads // kv
    tok = torch.arange(total, device=q.device)
    seq = torch.searchsorted(s["start"][1:].long(), tok, right=True)
    at = tok - s["start"].long()[seq]
    where = torch.arange(length, device=q.device)
    slot = s["table"].long()[:, where // page] * page + where % page          # (n, length)
    k, v = (c.flatten(0, 1)[slot].float() for c in (kc, vc))                  # (n, length, kv, dim)
    pad = q.new_zeros((n, most, heads, dim), dtype=torch.float32)
    pad[seq, at] = q.float()
    qs = pad.view(n, most, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, most * group, dim)
    score = qs @ k.permute(0, 2, 3, 1) * dim ** -0.5                          # (n, kv, most*group, length)
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
    o = torch.where(z > 0, (e @ v.permute(0, 2, 1, 3)) / z, torch.zeros_like(z))
    lse = torch.where(z > 0, top + torch.log(z), torch.full_like(z, -math.inf))
    o, lse = (x.view(n, kv, most, group, -1).permute(0, 2, 1, 3, 4).reshape(n, most, heads, -1)[seq, at] for x in (o, lse))
    return {"out": o.to(q.dtype), "lse": lse[..., 0]}


def _plain_sample(s):
    x = s["logits"].double()
    n, vocab = x.shape
    greedy = s["temperature"] == 0
    t = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()[:, None]
    sx, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((sx - sx[:, :1]) / t)
    rank = torch.arange(vocab, device=x.device)[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), vocab)[:, None]
    keep = (rank < k) & (w > 0)
    w = w * keep
    before = torch.cumsum(w, 1) - w
    keep &= (before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True)) | (s["top_p"] >= 1)[:, None]
    keep &= (w >= s["min_p"].double()[:, None]) | (rank == 0)
    by_index = torch.zeros_like(w).scatter_(1, order, w * keep)
    run_sum = torch.cumsum(by_index, 1)
    mass = run_sum[:, -1:]
    i = (run_sum <= s["u"].double()[:, None] * mass).sum(1, keepdim=True).clamp_max(vocab - 1)
    p = by_index.gather(1, i) / mass
    i, p = torch.where(greedy[:, None], order[:, :1], i), torch.where(greedy[:, None], torch.ones_like(p), p)
    return {"ids": i[:, 0].int(), "probs": p[:, 0].float()}


def run(s):
    c = s["case"]
    if own:
        from verify_matvec_gb300 import cbq
        if c["op"] == "rope":
            return cbq.cbq_rope(s["x"], s["pos"], s["turns"], rot_off=c["off"], layout=c["layout"], mscale=s["magnitude"])
        if c["op"] == "append":
            q = cbq.cbq_rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["turns"], s["kc"], s["vc"],
                                    rot_off=c["off"], layout=c["layout"], mscale=s["magnitude"])
            return {"q": q, "kc": s["kc"], "vc": s["vc"]}
        if c["op"] == "attn":
            out, lse = cbq.cbq_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["start"], s["mask"],
                                              max_tok=s["max_tok"], max_len=s["max_len"], with_lse=True)
            return {"out": out, "lse": lse}
        ids, probs = cbq.cbq_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"])
        return {"ids": ids, "probs": probs}
    if c["op"] == "rope":
        return _rotate(s, s["x"]).to(s["x"].dtype)
    if c["op"] == "append":
        s["kc"].flatten(0, 1)[s["slots"]] = _rotate(s, s["k"]).to(s["kc"].dtype)
        s["vc"].flatten(0, 1)[s["slots"]] = s["v"].to(s["vc"].dtype)
        return {"q": _rotate(s, s["q"]).to(s["kc"].dtype), "kc": s["kc"], "vc": s["vc"]}
    return _plain_attention(s) if c["op"] == "attn" else _plain_sample(s)


def work(case):
    d = SIZE[case["dtype"]]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * d + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        n, both = case["tokens"] * case["dim"], case["heads"] + 2 * case["kv"]
        return {"bytes": n * both * (d + SIZE[case["cache"]]) + 12 * case["tokens"],
                "flops": 3 * case["tokens"] * case["rot"] * (case["heads"] + case["kv"])}
    if case["op"] == "attn":
        keys = sum(c + n for c, n in _lengths(case))
        toks = sum(n for _, n in _lengths(case))
        pairs = sum((c + n) * n for c, n in _lengths(case))
        return {"bytes": 2 * keys * case["kv"] * case["dim"] * d + toks * case["heads"] * (2 * case["dim"] * d + 4),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    return {"bytes": case["rows"] * (case["vocab"] * d + 28), "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------- definitions in 64 bits --

def _turned(s, x):
    """The rotation as a product of complex numbers."""
    c = s["case"]
    x = x.double().cpu().numpy()
    t = s["pos"].double().cpu().numpy()[:, None] * s["turns"].cpu().numpy()[None, :]
    z = s["magnitude"] * np.exp(2j * np.pi * (t - np.floor(t)))[:, None, :]
    part = x[..., c["off"]:c["off"] + c["rot"]]
    shape = part.shape[:-1]
    two = part.reshape(*shape, 2, -1) if c["layout"] == "half" else np.swapaxes(part.reshape(*shape, -1, 2), -1, -2)
    r = (two[..., 0, :] + 1j * two[..., 1, :]) * z
    both = np.stack([r.real, r.imag], -2 if c["layout"] == "half" else -1).reshape(*shape, -1)
    out = x.copy()
    out[..., c["off"]:c["off"] + c["rot"]] = both
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s, s["x"])
    if case["op"] == "append":
        kc, vc = s["kc"].double().cpu().numpy(), s["vc"].double().cpu().numpy()
        for cache, new in ((kc, _turned(s, s["k"])), (vc, s["v"].double().cpu().numpy())):
            cache.reshape(-1, case["kv"], case["dim"])[s["slots"].cpu().numpy()] = new
        return {"q": _turned(s, s["q"]), "kc": kc, "vc": vc}
    if case["op"] == "attn":
        if work(case)["flops"] > 5e12:
            return None
        start, ctx, group = s["start"].tolist(), s["ctx"].tolist(), case["heads"] // case["kv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for i, c in enumerate(ctx):
            a, b = start[i], start[i + 1]
            pages = s["table"][i, :-(-(c + b - a) // case["page"])].long()
            allow = torch.ones(b - a, c + b - a, dtype=torch.bool, device="cuda")
            for j, m in enumerate(s["mask"][a:b].tolist()):
                allow[j, c:] = torch.tensor([bool(m >> x & 1) for x in range(b - a)], device="cuda")
            for h in range(case["heads"]):
                k, v = (x[pages, :, h // group].flatten(0, 1)[:c + b - a].double() for x in (s["kc"], s["vc"]))
                e = (s["q"][a:b, h].double() @ k.T / math.sqrt(case["dim"])).masked_fill(~allow, -math.inf)
                lse[a:b, h] = torch.logsumexp(e, 1)
                out[a:b, h] = torch.exp(e - lse[a:b, h, None]) @ v
        return {"out": out, "lse": lse}
    ids, probs = [], []
    for i, row in enumerate(s["logits"].double().cpu().numpy()):
        t, k, p, m, u = (float(s[x][i]) for x in ("temperature", "top_k", "top_p", "min_p", "u"))
        order = np.lexsort((np.arange(row.size), -row))
        if t == 0:
            ids.append(int(order[0]))
            probs.append(1.0)
            continue
        order = order[:int(k)] if k else order
        w = np.exp((row[order] - row[order[0]]) / t)
        sums = np.cumsum(w)
        kept = order.size if p >= 1 else int(np.searchsorted(sums, p * sums[-1])) + 1
        kept = max(1, min(kept, int(np.sum(w >= m))))
        chosen = np.argsort(order[:kept])
        sums = np.cumsum(w[chosen])
        j = chosen[min(int(np.searchsorted(sums, u * sums[-1], side="right")), kept - 1)]
        ids.append(int(order[j]))
        probs.append(float(w[j] / sums[-1]))
    return {"ids": np.array(ids, np.int32), "probs": np.array(probs)}
