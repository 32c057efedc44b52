"""The operators together, as the example runs them: one verify step against
the definitions in 64 bits, each from the values the step before it gave."""
import importlib.util
import os

import numpy as np
import pytest

from tests import step_ref
from tests.conftest import ROOT
from tests.gpu_util import cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.fixture(scope="module")
def example(torch):
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_verify_step(torch, example):
    layer = example.Layer()
    g = torch.Generator(device="cuda").manual_seed(3)
    for c in (layer.kc, layer.vc):
        c.normal_(generator=g)
    ctx, parents = 45, [-1, 0, 1, 0, 3]
    n, h, kv, d = 5, layer.heads, layer.kv, layer.dim
    table = torch.randperm(32, generator=g, device="cuda")[:8].to(torch.int32)[None]
    x = torch.randn((n, layer.hidden), generator=g, device="cuda")
    t, p = torch.full((n,), 0.8, device="cuda"), torch.full((n,), 0.95, device="cuda")
    k, u = torch.full((n,), 50, dtype=torch.int32, device="cuda"), torch.rand(n, generator=g, device="cuda")
    before = layer.kc.clone(), layer.vc.clone()
    r = example.verify_step(layer, x, ctx, parents, table, t, k, p, u)

    num = lambda y: y.double().cpu().numpy()  # noqa: E731
    qkv = num(cbq.cbq_matvec(layer.qkv, x)).reshape(n, h + 2 * kv, d)
    pos = np.array([45, 46, 47, 46, 47])
    turns = num(layer.turns)
    wq, _ = step_ref.rotate(qkv[:, :h], pos, turns, 0, "half")
    wk, _ = step_ref.rotate(qkv[:, h:h + kv], pos, turns, 0, "half")
    # one bf16 rounding (2^-8 with the fp32 arithmetic's share)
    assert np.all(np.abs(num(r["q"]) - wq) <= np.abs(wq) * 2.0 ** -8 + 1e-6)
    place = np.arange(ctx, ctx + n)
    pages = table[0].cpu().numpy()[place // 16]
    kc, vc = num(layer.kc), num(layer.vc)
    assert np.all(np.abs(kc[pages, place % 16] - wk) <= np.abs(wk) * 2.0 ** -8 + 1e-6)
    assert np.all(np.abs(vc[pages, place % 16] - qkv[:, h + kv:]) <= np.abs(qkv[:, h + kv:]) * 2.0 ** -8)
    same = np.ones(kc.shape[:2], dtype=bool)
    same[pages, place % 16] = False
    assert np.array_equal(kc[same], num(before[0])[same]) and np.array_equal(vc[same], num(before[1])[same])
    mask = np.array([1, 3, 7, 9, 25])
    out, _, absv, _ = step_ref.attention(num(r["q"]), kc, vc, table.cpu().numpy(), [ctx], [0, n], mask, d ** -0.5)
    assert np.all(np.abs(num(r["att"]) - out) <= absv * 2.0 ** -8 + 1e-6)
    logits = num(r["logits"])
    for i in range(n):
        want, prob, margin = step_ref.sample(logits[i], float(t[i]), 50, float(p[i]), 0.0, float(u[i]))
        assert margin < 2.0 ** -30 or (int(r["ids"][i]) == want and abs(float(r["probs"][i]) - prob) <= 2.0 ** -23 * prob)
    assert example.accepted(r["ids"].tolist(), [0, int(r["ids"][0]), -1, 0, 0], parents)[:2] == [0, 1]
