"""libcbq.so as a C program has it: in a process without PyTorch, on a machine
that has the driver and no CUDA toolkit."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tests.conftest import ROOT
from tests.gpu_util import assert_within_bound, cuda
from verify_matvec_gb300 import build

ALONE = dict(os.environ, LD_LIBRARY_PATH="", PYTHONPATH=ROOT)


def _run(code, *args):
    r = subprocess.run([sys.executable, "-c", code, build.build(), *args], env=ALONE, cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


LOADED = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
lib.cbq_status_string.restype = ctypes.c_char_p
assert lib.cbq_status_string(0).startswith(b"CBQ_")
assert lib.cbq_quantize_act(None, ctypes.c_int64(64), 1, None, None, None) == -1
with open("/proc/self/maps") as f:
    maps = f.read()
assert "libcudart" not in maps and "torch" not in maps, "brings another library of the toolkit"
"""


def test_needs_no_library_of_the_toolkit():
    out = subprocess.run(["readelf", "-d", build.build()], capture_output=True, text=True, check=True).stdout
    needed = [line.split("[")[1].rstrip("]") for line in out.splitlines() if "NEEDED" in line]
    own = ("libstdc++.", "libm.", "libgcc_s.", "libc.", "ld-linux", "libdl.", "libpthread.", "librt.")
    assert needed and all(n.startswith(own) for n in needed), needed
    assert "RUNPATH" not in out and "RPATH" not in out, "looks into this machine's folders"
    _run(LOADED)


@pytest.mark.gpu
def test_runs_alone(tmp_path):
    cuda()
    from oracle import oracle as O
    from verify_matvec_gb300 import synth
    M, K, n = 96, 256, 3
    blocks, x = synth.weight_blocks(M, K, stream=41), synth.activations(n, K, stream=42)
    np.save(tmp_path / "b.npy", blocks)
    np.save(tmp_path / "x.npy", x)
    _run(LOADED + f"""
import numpy as np
P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
b, x = (np.load(p) for p in sys.argv[2:4])
y, h = np.zeros(({n}, {M}), np.float32), P()
rc = lib.cbq_weights_create(P(b.ctypes.data), L({M}), L({K}), I(0), None, ctypes.byref(h))
assert rc == 0, rc
rc = lib.cbq_matvec_host(h, P(x.ctypes.data), I({n}), P(y.ctypes.data), None)
assert rc == 0, rc
assert lib.cbq_weights_destroy(h) == 0
with open("/proc/self/maps") as f:
    assert "libcudart" not in f.read()
np.save(sys.argv[4], y)
""", str(tmp_path / "b.npy"), str(tmp_path / "x.npy"), str(tmp_path / "y.npy"))
    qx, dx = O.quantize_act(x)
    assert_within_bound(np.load(tmp_path / "y.npy"), O.matvec(blocks, M, K, x), O.matvec_bound(blocks, M, K, qx, dx))
