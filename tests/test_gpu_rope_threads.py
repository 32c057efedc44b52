"""Rotations of different sizes from two host threads at a time, each on its
own stream: neither call's shared memory is the other's limit."""
import threading

import pytest

from tests.gpu_util import cuda
from verify_matvec_gb300 import cbq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return cuda()


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_two_sizes_at_once(torch, layout):
    n, calls = 5000, 4000  # (tokens enough for the blocks that go through several)
    failed, start = [], threading.Barrier(2)

    def worker(rot):
        try:
            stream = torch.cuda.Stream()
            x = torch.randn((n, 1, rot), device="cuda").bfloat16()
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            turns, out = cbq.cbq_rope_turns(rot), torch.empty_like(x)
            want = cbq.cbq_rope(x, pos, turns, layout=layout)
            torch.cuda.synchronize()
            start.wait()
            for _ in range(calls):
                cbq.cbq_rope(x, pos, turns, layout=layout, out=out, stream=stream)
            stream.synchronize()
            assert torch.equal(out, want)
        except Exception as e:  # noqa: BLE001
            failed.append((rot, e))

    threads = [threading.Thread(target=worker, args=(rot,)) for rot in (64, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
