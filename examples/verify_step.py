"""One verify step of speculative decoding through the library: a tree of
drafted tokens goes through one decoder layer and the output head, and either a
token is drawn at each of them, or the tree is verified against what its drafts
were drawn from and the cache brought up to date.

    x (tokens x hidden)
      -> cbq_matvec            q, k, v of the drafts (codebook-4bit weights)
      -> cbq_rope_append       rotary positions; k, v into the paged cache
      -> cbq_tree_attention    each draft over the context and its ancestors
      -> cbq_matvec            output projection, residual
      -> cbq_moe_matvec_logits routed experts, residual
      -> cbq_matvec            logits
      -> cbq_sample            one token a draft
    or
      -> cbq_probs             the target's and the drafter's distributions
      -> cbq_verify            the accepted drafts and the token behind them
      -> cbq_kv_commit         their keys and values to the end of the context

Run it: python examples/verify_step.py  (random weights; needs the GPU).
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from verify_matvec_gb300 import cbq, synth  # noqa: E402


class Layer:
    """One layer's weights and its cache: `pages` pages of `page` tokens."""

    def __init__(self, hidden=512, heads=8, kv=2, dim=64, experts=8, inner=256, vocab=4000, pages=32, page=16):
        self.hidden, self.heads, self.kv, self.dim, self.page, self.topk = hidden, heads, kv, dim, page, 2
        blocks = lambda m, k, stream, hi=1e-3: synth.weight_blocks(m, k, stream=stream, scale_lo=1e-5, scale_hi=hi)  # noqa: E731
        W = lambda m, k, *a: cbq.Weights(blocks(m, k, *a), m, k)  # noqa: E731
        self.qkv = W((heads + 2 * kv) * dim, hidden, 801)
        self.o = W(hidden, heads * dim, 802)
        self.router = W(experts, hidden, 803)
        self.moe = cbq.Moe(np.stack([blocks(2 * inner, hidden, 810 + e) for e in range(experts)]),
                           np.stack([blocks(hidden, inner, 830 + e) for e in range(experts)]), experts, hidden, inner)
        self.head = W(vocab, hidden, 804, 3e-3)
        self.turns = cbq.cbq_rope_turns(dim)
        self.kc, self.vc = (torch.zeros((pages, page, kv, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")


def verify_step(layer, x, ctx, parents, table, temperature, top_k, top_p, u):
    """x (tokens, hidden) fp32 of the drafts; ctx committed tokens in the cache;
    parents[i] the index of draft i's parent among them (-1: the context);
    table (1, width) int32 the sequence's pages.  Returns what the step drew
    (ids, probs), with the attention's output and the logits."""
    n, dev = x.shape[0], x.device
    depth, bits = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        bits.append((0 if p < 0 else bits[p]) | 1 << i)
    place = torch.arange(ctx, ctx + n, device=dev)
    slots = table[0, place // layer.page].long() * layer.page + place % layer.page
    pos = torch.tensor([ctx + d for d in depth], dtype=torch.int32, device=dev)

    h, kv, d = layer.heads, layer.kv, layer.dim
    qkv = cbq.cbq_matvec(layer.qkv, x).view(n, h + 2 * kv, d)
    q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    q = cbq.cbq_rope_append(q, k, v, pos, slots, layer.turns, layer.kc, layer.vc)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    att = torch.empty((n, h, d), dtype=torch.float32, device=dev)
    cbq.cbq_tree_attention(q, layer.kc, layer.vc, table, i32([ctx]), i32([0, n]),
                           torch.tensor(bits, dtype=torch.int64, device=dev), max_tok=n, max_len=ctx + n, out=att)
    x = x + cbq.cbq_matvec(layer.o, att.view(n, h * d))
    x = x + cbq.cbq_moe_matvec_logits(layer.moe, x, cbq.cbq_matvec(layer.router, x), layer.topk)
    logits = cbq.cbq_matvec(layer.head, x)
    ids, probs = cbq.cbq_sample(logits, temperature, top_k, top_p, None, u)
    return {"ids": ids, "probs": probs, "q": q, "att": att, "logits": logits}


def accepted(ids, drafts, parents):
    """The drafts that the step confirms: from the root on, the child that is the token drawn at its parent."""
    path, at = [], 0
    while True:
        path.append(at)
        at = next((i for i, p in enumerate(parents) if p == at and drafts[i] == ids[at]), None)
        if at is None:
            return path


def settle(layer, ctx, parents, table, tokens, logits, drafter, temperature, top_k, top_p, u, u_next):
    """What stays of a step's drafts, so that what comes out is distributed as
    the target's own tokens: logits (nodes, V) of the step, drafter (nodes, V)
    the logits from which each node's children were drawn, with the same
    temperature and cuts, tokens (nodes) int32 the drafts (node 0's is settled
    already).  The cache keeps the accepted nodes behind the context.  Returns
    path and count (the accepted nodes), the next token and the new length."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=logits.device)  # noqa: E731
    n = logits.shape[0]
    probs = cbq.cbq_probs(logits, temperature, top_k, top_p, None)
    draft = cbq.cbq_probs(drafter, temperature, top_k, top_p, None)
    path, count, token = cbq.cbq_verify(probs, draft, tokens, i32(parents), i32([0, n]), u, u_next, n)
    length = cbq.cbq_kv_commit(layer.kc, layer.vc, table, i32([ctx]), path, count)
    return {"path": path, "count": count, "token": token, "length": length, "probs": probs, "draft": draft}


def main():
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    # draft 0 is the last committed token's successor; two branches hang off it
    ctx, parents = 45, [-1, 0, 1, 0, 3]
    n = len(parents)
    for c in (layer.kc, layer.vc):
        c.normal_(generator=g)
    table = torch.randperm(32, generator=g, device="cuda")[:8].to(torch.int32)[None]
    x = torch.randn((n, layer.hidden), generator=g, device="cuda")
    f = lambda v, t: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    r = verify_step(layer, x, ctx, parents, table, f(0.8, torch.float32), f(50, torch.int32), f(0.95, torch.float32),
                    torch.rand(n, generator=g, device="cuda"))
    ids = r["ids"].tolist()
    drafts = [0, ids[0], ids[1], 7, 9]  # (as if the drafter had guessed the first branch)
    print("drawn", ids, "probabilities", [round(p, 3) for p in r["probs"].tolist()])
    print("accepted drafts", accepted(ids, drafts, parents))
    # the same step's tree as a drafter's own draws: its logits are near the target's
    drafter = r["logits"] + 0.3 * torch.randn(r["logits"].shape, generator=g, device="cuda")
    cuts = (f(0.8, torch.float32), f(50, torch.int32), f(0.95, torch.float32))
    drawn = torch.zeros(n, dtype=torch.int32, device="cuda")
    for i, p in enumerate(parents):
        if p >= 0:
            drawn[i] = cbq.cbq_sample(drafter[p:p + 1], *(c[:1] for c in cuts), None, torch.rand(1, generator=g, device="cuda"))[0][0]
    s = settle(layer, ctx, parents, table, drawn, r["logits"], drafter, *cuts, torch.rand(n, generator=g, device="cuda"),
               torch.rand(1, generator=g, device="cuda"))
    print("verified: nodes", s["path"][0].tolist(), "next token", s["token"].item(), "context", s["length"].item())


if __name__ == "__main__":
    main()
