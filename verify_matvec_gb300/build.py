"""Build libcbq.so (the C-ABI library) in-tree with nvcc for sm_103a.

The translation units are compiled in parallel and linked twice, next to this
file:
  libcbq.so          with the CUDA runtime inside, for C programs: it needs
                     the driver and nothing of the toolkit;
  libcbq_binding.so  the same objects with the shared runtime, which the
                     binding loads: PyTorch has brought it already, and one
                     runtime's code and not two is worth 3 us a call where
                     tensor operations and the library's calls take turns (an
                     allocation and a launch 9.4 us with a runtime of the
                     library's own, 6.1 so).
`python -m verify_matvec_gb300.build` or `build()`, which returns the path of
libcbq.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libcbq.so")
OUT_BINDING = os.path.join(HERE, "libcbq_binding.so")
OBJDIR = os.path.join(HERE, "_build")
SOURCES = ["cbq_kernels.cu", "cbq_mmq.cu", "cbq_hc.cu", "cbq_rope.cu", "cbq_attn.cu", "cbq_attn_wide.cu", "cbq_sample.cu", "cbq_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-v", "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcbq.so")


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _stale() -> bool:
    if not (os.path.exists(OUT) and os.path.exists(OUT_BINDING)):
        return True
    t = min(os.path.getmtime(OUT), os.path.getmtime(OUT_BINDING))
    deps = [os.path.join(d, f) for d, _, files in os.walk(CSRC) for f in files]
    deps += [os.path.join(INCLUDE, "cbq.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _link(out: str, objs: list[str], *how: str):
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, *how], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return OUT
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(_compile, SOURCES))
    objs = [o for o, _ in results]
    log = "\n".join(e for _, e in results)
    with open(os.path.join(OBJDIR, "ptxas.log"), "w") as f:
        f.write(log)
    if verbose:
        print(log)
    libs = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "lib64")
    _link(OUT, objs, "-cudart", "static")
    _link(OUT_BINDING, objs, "-cudart", "shared", "-Xlinker", "-rpath," + libs)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
