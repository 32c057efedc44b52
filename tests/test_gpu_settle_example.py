"""The example's end of a verify step: the distributions, the verification of a
tree and the cache behind it, against the definitions in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.fixture(scope="module")
def example(torch):
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_settle(torch, example):
    layer = example.Layer()
    g = torch.Generator(device="cuda").manual_seed(8)
    for c in (layer.kc, layer.vc):
        c.normal_(generator=g)
    ctx, parents = 45, [-1, 0, 1, 0, 3, 3]
    n, V = len(parents), 4000
    table = torch.randperm(32, generator=g, device="cuda")[:8].to(torch.int32)[None]
    for near in (0.05, 0.5, 4.0):
        logits = torch.randn((n, V), generator=g, device="cuda") * 2
        drafter = logits + near * torch.randn((n, V), generator=g, device="cuda")
        full = lambda v, t=torch.float32: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
        cuts = full(0.8), full(50, torch.int32), full(0.95)
        tokens = torch.tensor([0] + [int(drafter[p].argmax()) if i != 4 else int(drafter[p].topk(2)[1][1]) for i, p in enumerate(parents) if p >= 0],
                              dtype=torch.int32, device="cuda")
        u, un = torch.rand(n, generator=g, device="cuda"), torch.rand(1, generator=g, device="cuda")
        bits = lambda x: x[None].view(torch.int16).cpu().numpy()  # noqa: E731
        before = bits(layer.kc), bits(layer.vc)
        r = example.settle(layer, ctx, parents, table, tokens, logits, drafter, *cuts, u, un)
        num = lambda y: y.double().cpu().numpy()  # noqa: E731
        for x, y in ((logits, r["probs"]), (drafter, r["draft"])):
            for i in range(n):
                want, margin = behind_ref.probs(num(x[i]), float(cuts[0][i]), 50, float(cuts[2][i]), 0.0)
                assert margin < 2.0 ** -30 or np.all(np.abs(num(y[i]) - want) <= 2.0 ** -23 * (1 + 2.0 ** -14) * want + 2.0 ** -45)
        path, token, margin = behind_ref.verify(num(r["probs"]), num(r["draft"]), tokens.tolist(), parents, u.tolist(), float(un))
        if margin >= 2.0 ** -40:
            assert r["path"][0].tolist() == path + [-1] * (n - len(path)) and r["token"].tolist() == [token]
        count = int(r["count"])
        assert r["length"].tolist() == [ctx + count]
        want = behind_ref.commit(*before, table.cpu().numpy(), [ctx], r["path"].cpu().numpy(), [count])
        assert np.array_equal(bits(layer.kc), want[0]) and np.array_equal(bits(layer.vc), want[1])
