"""Ends of what the calls behind the logits allow: rows and pages whose places
pass 32 bits, numbers u outside [0, 1), contexts of nothing, and the same page
read by two sequences."""
import numpy as np
import pytest

from tests import behind_ref
from tests.gpu_util import cuda
from tests.test_gpu_tree_attention8 import Setup
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


def _far(torch, like, stride):
    """A tensor like `like` whose first axis has that stride; nothing in between is written."""
    n = like.shape[0]
    inner = like[0].numel()
    room = torch.empty((n - 1) * stride + inner, dtype=like.dtype, device="cuda")
    out = room.as_strided(like.shape, (stride, *like[0].contiguous().stride()))
    out.copy_(like)
    return out


@pytest.mark.parametrize("V", [1000, 1001])
def test_rows_far_apart(torch, V):
    """Rows more than 2^31 values from the first: as those side by side."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((3, V), generator=g, device="cuda")
    top = torch.full((3,), 0.9, device="cuda")
    p = cbq.cbq_probs(x, None, None, top, None)
    d = cbq.cbq_probs(x + torch.randn((3, V), generator=g, device="cuda"), None, None, None, None)
    far = _far(torch, torch.zeros_like(p), (1 << 30) + 16)
    assert torch.equal(cbq.cbq_probs(_far(torch, x, (1 << 30) + 16), None, None, top, None, out=far), p)
    assert torch.equal(far, p)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tokens = torch.cat([i32(0), d[:2].argmax(1).int()])
    for u in (0.0, 0.5, 0.999):
        rest = (tokens, i32(-1, 0, 1), i32(0, 3), torch.full((3,), u, device="cuda"), torch.full((1,), u, device="cuda"), 3)
        want = cbq.cbq_verify(p, d, *rest)
        for near in ((far, d), (far, _far(torch, d, (1 << 30) + 16))):
            assert all(torch.equal(a, b) for a, b in zip(cbq.cbq_verify(*near, *rest), want))


@pytest.mark.parametrize("heads,drafts,dim", [(4, 1, 128), (8, 20, 64), (8, 40, 128), (4, 2, 72)])
def test_pages_far_apart(torch, heads, drafts, dim):
    """Pages more than 2^32 bytes from the first, of both caches."""
    s = Setup(torch, [70], [20], [drafts], heads, 1, dim, 48, 48, 16, seed=dim)
    out, lse = s.run()
    s.k8, s.v8, s.kc, s.vc = (_far(torch, x, (1 << 31) + 256) for x in (s.k8, s.v8, s.kc, s.vc))
    out2, lse2 = s.run()
    assert int(s.err) == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)
    s.check(out2, lse2)


def test_pages_far_apart_are_written(torch):
    """Moves and 8-bit pages more than 2^32 bytes from the first; layers too."""
    g = torch.Generator(device="cuda").manual_seed(9)
    kc, vc = (torch.randn((3, 16, 2, 64), generator=g, device="cuda").bfloat16() for _ in "kv")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    path = i32(1, 3, 20, -1)[None]
    want = behind_ref.commit(*(x[None].view(torch.int16).cpu().numpy() for x in (kc, vc)), np.array([[2, 1, 0]]), [14], [[1, 3, 20, -1]], [3])
    far = [_far(torch, x, (1 << 31) + 256) for x in (kc, vc)]
    path = torch.nn.functional.pad(path, (0, 28), value=-1)
    err = i32(0)
    new = cbq.cbq_kv_commit(*far, i32(2, 1, 0)[None], i32(14), path, i32(3), err=err)
    assert new.tolist() == [17] and int(err) == 0
    for x, w in zip(far, want):
        assert np.array_equal(x.contiguous().view(torch.int16).cpu().numpy(), w[0])
    # as two layers far apart, of one page each
    layers = [x[1:].unsqueeze(1) for x in far]
    k8, v8 = (_far(torch, torch.zeros((2, 1, 16, 2, 64), dtype=torch.uint8, device="cuda"), (1 << 32) + 256).view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros((2, 1, 2, 2), device="cuda") for _ in "kv")
    cbq.cbq_kv_quantize(*layers, i32(0), k8, v8, ks, vs, i32(0), err=err)
    for x, x8, scale in ((layers[0], k8, ks), (layers[1], v8, vs)):
        for y in range(2):
            number, of = behind_ref.quantize(x[y].double().cpu().numpy(), 8)
            assert np.array_equal(x8[y].double().cpu().numpy(), number) and np.array_equal(scale[y].double().cpu().numpy(), of)
    assert int(err) == 0


def test_numbers_outside(torch):
    """u of NaN accepts nothing, one below 0 whatever has a share; u_next is held inside [0, 1)."""
    V = 300
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.softmax(torch.randn((2, V), generator=g, device="cuda"), 1)
    p[:, :5] = 0
    p[:, -7:] = 0
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    nan, inf = float("nan"), float("inf")
    for u, took in ((nan, 0), (-1.0, 1), (inf, 0)):
        for un, end in ((nan, 0), (-3.0, 0), (1.0, 1), (inf, 1)):
            path, count, token = cbq.cbq_verify(p, p, i32(0, 50), i32(-1, 0), i32(0, 2), torch.full((2,), u, device="cuda"),
                                                torch.full((1,), un, device="cuda"), 2)
            assert int(count) == 1 + took, (u, un)
            # (where the draft equals the target and was refused, the token is drawn from the target)
            assert int(token) == (V - 8 if end else 5), (u, un, int(token))


def test_one_page_of_two_sequences(torch):
    """Two sequences over the same 8-bit pages and the same pages behind them see what each would alone."""
    s = Setup(torch, [64, 64], [3, 3], [2, 2], 8, 2, 128, 16, 16, 16, seed=2)
    s.table8[1] = s.table8[0]
    s.table[1] = s.table[0]
    out, lse = s.run()
    s.check(out, lse)
    assert int(s.err) == 0
