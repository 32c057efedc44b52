"""Thin ctypes binding of libcbq.so (include/cbq.h), same names as the C ABI.

Argument marshalling only: torch tensors give device pointers and the current
stream, numpy arrays give host pointers.  Every step of the path runs in the
library's CUDA kernels; if the library is missing this module raises instead of
computing anything another way.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcbq_binding.so")  # libcbq.so on the CUDA runtime that PyTorch has loaded
HEADER = os.path.join(os.path.dirname(HERE), "include", "cbq.h")

CBQ_OK, CBQ_EINVAL, CBQ_ECUDA, CBQ_ENOMEM, CBQ_EDEVICE = 0, -1, -2, -3, -4
CBQ_QK = 32
CBQ_BLOCK_BYTES = 18
CBQ_MAX_COLS = 5
CBQ_MAX_TOKENS = 5
CBQ_MAX_TOPK = 16
CBQ_DEVERR_BAD_EXPERT_ID = 0x1
CBQ_DEVERR_PIPE_TIMEOUT = 0x100
CBQ_DEVERR_DEPENDENCY_TIMEOUT = 0x200
CBQ_STATIC_SCRATCH_MAX_K = 16384
CBQ_ROUTER_MAX_E = 16384
CBQ_MAX_MMQ_COLS = 16
CBQ_HC_NHC = 4
CBQ_HC_MAX_ITERS = 1024
CBQ_HC_MAX_N = 1 << 28
CBQ_F32, CBQ_BF16, CBQ_F16 = 0, 1, 2
CBQ_DEVERR_BAD_SLOT = 0x2
CBQ_DEVERR_BAD_LENGTH = 0x4
CBQ_ROPE_NONE, CBQ_ROPE_LINEAR, CBQ_ROPE_BY_TURNS, CBQ_ROPE_BY_INDEX = 0, 1, 2, 3
CBQ_ROPE_HALF, CBQ_ROPE_PAIRS = 0, 1
CBQ_ROPE_MAX_DIM = 1024
CBQ_TREE_MAX = 64
CBQ_TREE_MAX_LEN = 1 << 30
CBQ_SAMPLE_MAX_V = 1 << 18

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_D = ctypes.c_double


class cbq_kv_cache(ctypes.Structure):
    """The C struct of the same name: a paged cache of keys and values."""
    _fields_ = [("k", _P), ("v", _P), ("dtype", _I), ("kv_heads", _I), ("head_dim", _I), ("page_size", _I),
                ("n_pages", _I64), ("page_stride", _I64), ("tok_stride", _I64), ("head_stride", _I64)]


_KV = ctypes.POINTER(cbq_kv_cache)
_SIGS = {
    "cbq_status_string": ([_I], ctypes.c_char_p),
    "cbq_last_cuda_error": ([], ctypes.c_char_p),
    "cbq_weights_create": ([_P, _I64, _I64, _I, _P, ctypes.POINTER(_P)], _I),
    "cbq_weights_destroy": ([_P], _I),
    "cbq_weights_info": ([_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)], _I),
    "cbq_quantize_act": ([_P, _I64, _I, _P, _P, _P], _I),
    "cbq_matvec_q": ([_P, _P, _P, _I, _P, _P], _I),
    "cbq_matvec": ([_P, _P, _I, _P, _P], _I),
    "cbq_matvec_host": ([_P, _P, _I, _P, _P], _I),
    "cbq_matvec_static": ([_P, _P, _I, _P, _P], _I),
    "cbq_moe_create": ([_P, _P, _I, _I64, _I64, _I, _P, ctypes.POINTER(_P)], _I),
    "cbq_moe_destroy": ([_P], _I),
    "cbq_moe_set_shared": ([_P, _P, _P, _I, _P], _I),
    "cbq_moe_info": ([_P, ctypes.POINTER(_I), ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)], _I),
    "cbq_moe_matvec": ([_P, _P, _I, _P, _P, _I, _I, _P, _P], _I),
    "cbq_moe_matvec_host": ([_P, _P, _I, _P, _P, _I, _I, _P, _P], _I),
    "cbq_router_topk": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "cbq_quantize_weights": ([_P, _I64, _I64, _P, _P], _I),
    "cbq_hc_sinkhorn": ([_P, _I64, _I, _P, _P], _I),
    "cbq_matmat": ([_P, _P, _I, _P, _P], _I),
    "cbq_debug_mmq_block_dots": ([_P, _P, _I, _P, _P], _I),
    "cbq_moe_matvec_logits": ([_P, _P, _I, _P, _I, _I, _P, _P], _I),
    "cbq_weights_get_error": ([_P, _P, ctypes.POINTER(ctypes.c_uint)], _I),
    "cbq_moe_get_error": ([_P, _P, ctypes.POINTER(ctypes.c_uint)], _I),
    "cbq_moe_debug_stall": ([_P, _I], _I),
    "cbq_debug_mmq_stall": ([_P, _I], _I),
    "cbq_debug_block_dots": ([_P, _P, _I, _P, _P], _I),
    "cbq_moe_debug_block_dots": ([_P, _I, _I, _P, _I, _P, _P], _I),
    "cbq_moe_set_debug": ([_P, _I], _I),
    "cbq_moe_set_stage_events": ([_P, _P, _P, _P], _I),
    "cbq_rope_turns": ([_I, _D, _I, _D, _D, _D, _D, _P], _I),
    "cbq_rope": ([_P, _I, _I64, _I, _I, _I64, _I64, _P, _P, _I, _I, _I, _F, _P, _I64, _I64, _P], _I),
    "cbq_rope_append": ([_P, _P, _P, _I, _I64, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _I, _I, _I, _F, _KV, _P, _P,
                         _P], _I),
    "cbq_tree_attention_workspace": ([_I, _I64, _I, _I64, _I, _I, _I, ctypes.POINTER(_I64)], _I),
    "cbq_tree_attention": ([_P, _I64, _I64, _I, _I64, _KV, _P, _I, _I, _P, _P, _P, _I, _I64, _F, _P, _I, _P, _P, _I64,
                            _P, _P], _I),
    "cbq_debug_tree_stall": ([_I], _I),
    "cbq_sample": ([_P, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "cbq_moe_debug_intermediate": ([_P, _I, _P, _P, _P, _P], _I),
}

_lib = None


class CbqError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.cbq_status_string(status).decode()
        cuda = lib.cbq_last_cuda_error().decode()
        super().__init__(f"{where}: {msg}" + (f" [{cuda}]" if cuda else ""))
        self.status = status


def header_functions() -> list[str]:
    """Names of the functions include/cbq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:int|const char \*)\s*(cbq_\w+)\s*\(", text, re.M)))


def load():
    """Load the library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m verify_matvec_gb300.build`; "
                          "this package has no CPU path")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != CBQ_OK:
        raise CbqError(status, where)


# ----------------------------------------------------------- marshalling --

def _torch():
    import torch
    return torch


def _dev_ptr(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _host_ptr(a: np.ndarray, dtype, name):
    if not isinstance(a, np.ndarray) or a.dtype != dtype or not a.flags["C_CONTIGUOUS"]:
        raise TypeError(f"{name} must be a C-contiguous numpy {np.dtype(dtype).name} array")
    return a.ctypes.data_as(ctypes.c_void_p)


# ----------------------------------------------------------------- handles --

class Weights:
    """cbq_weights: one dense M x K codebook-4bit matrix on the device."""

    def __init__(self, blocks, M: int, K: int, stream=None):
        torch = _torch()
        lib = load()
        h = ctypes.c_void_p()
        if isinstance(blocks, torch.Tensor):
            if blocks.numel() != M * (K // CBQ_QK) * CBQ_BLOCK_BYTES:
                raise ValueError("blocks do not match M x K")
            ptr, on_dev = _dev_ptr(blocks, torch.uint8, "blocks"), 1
        else:
            blocks = np.ascontiguousarray(blocks, dtype=np.uint8)
            if blocks.size != M * (K // CBQ_QK) * CBQ_BLOCK_BYTES:
                raise ValueError("blocks do not match M x K")
            ptr, on_dev = blocks.ctypes.data_as(ctypes.c_void_p), 0
        _check(lib.cbq_weights_create(ptr, M, K, on_dev, _stream(stream), ctypes.byref(h)), "cbq_weights_create")
        self._h = h
        self.M, self.K = M, K

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("destroyed handle")
        return self._h

    def device_bytes(self) -> int:
        b = ctypes.c_int64()
        _check(load().cbq_weights_info(self.handle, None, None, ctypes.byref(b)), "cbq_weights_info")
        return b.value

    def close(self):
        if getattr(self, "_h", None) is not None:
            load().cbq_weights_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Moe:
    """cbq_moe: E experts, each a stacked gate_up (2F x H) and a down (H x F)."""

    def __init__(self, gate_up, down, E: int, H: int, F: int, stream=None):
        torch = _torch()
        lib = load()
        h = ctypes.c_void_p()
        if isinstance(gate_up, torch.Tensor):
            p1, p2, on_dev = _dev_ptr(gate_up, torch.uint8, "gate_up"), _dev_ptr(down, torch.uint8, "down"), 1
        else:
            gate_up = np.ascontiguousarray(gate_up, dtype=np.uint8)
            down = np.ascontiguousarray(down, dtype=np.uint8)
            p1, p2, on_dev = gate_up.ctypes.data_as(_P), down.ctypes.data_as(_P), 0
        nbH, nbF = H // CBQ_QK, F // CBQ_QK
        n_gu = gate_up.numel() if isinstance(gate_up, torch.Tensor) else gate_up.size
        n_dn = down.numel() if isinstance(down, torch.Tensor) else down.size
        if n_gu != E * 2 * F * nbH * CBQ_BLOCK_BYTES or n_dn != E * H * nbF * CBQ_BLOCK_BYTES:
            raise ValueError("expert blocks do not match E, H, F")
        _check(lib.cbq_moe_create(p1, p2, E, H, F, on_dev, _stream(stream), ctypes.byref(h)), "cbq_moe_create")
        self._h = h
        self.E, self.H, self.F = E, H, F
        self.shared = False

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("destroyed handle")
        return self._h

    def set_shared(self, gate_up, down, stream=None):
        """cbq_moe_set_shared: a shared expert of the layer's shapes (blocks of
        one gate_up 2F x H and one down H x F), or None, None to remove it."""
        if (gate_up is None) != (down is None):
            raise ValueError("pass both gate_up and down blocks, or neither to remove the shared expert")
        torch = _torch()
        lib = load()
        if gate_up is None:
            _check(lib.cbq_moe_set_shared(self.handle, None, None, 0, _stream(stream)), "cbq_moe_set_shared")
            self.shared = False
            return
        nbH, nbF = self.H // CBQ_QK, self.F // CBQ_QK
        if isinstance(gate_up, torch.Tensor):
            p1, p2, on_dev = _dev_ptr(gate_up, torch.uint8, "gate_up"), _dev_ptr(down, torch.uint8, "down"), 1
            n_gu, n_dn = gate_up.numel(), down.numel()
        else:
            gate_up = np.ascontiguousarray(gate_up, dtype=np.uint8)
            down = np.ascontiguousarray(down, dtype=np.uint8)
            p1, p2, on_dev = gate_up.ctypes.data_as(_P), down.ctypes.data_as(_P), 0
            n_gu, n_dn = gate_up.size, down.size
        if n_gu != 2 * self.F * nbH * CBQ_BLOCK_BYTES or n_dn != self.H * nbF * CBQ_BLOCK_BYTES:
            raise ValueError("shared expert blocks do not match H, F")
        _check(lib.cbq_moe_set_shared(self.handle, p1, p2, on_dev, _stream(stream)), "cbq_moe_set_shared")
        self.shared = True

    def device_bytes(self) -> int:
        b = ctypes.c_int64()
        _check(load().cbq_moe_info(self.handle, None, None, None, ctypes.byref(b)), "cbq_moe_info")
        return b.value

    def close(self):
        if getattr(self, "_h", None) is not None:
            load().cbq_moe_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------- entry points --

def cbq_quantize_act(x, qx=None, dx=None, stream=None):
    """x: (n, K) float32 CUDA tensor -> (qx int8 (n, K), dx float32 (n, K/32))."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    n, K = x2.shape
    if qx is None:
        qx = torch.empty((n, K), dtype=torch.int8, device=x.device)
    if dx is None:
        dx = torch.empty((n, K // CBQ_QK), dtype=torch.float32, device=x.device)
    _check(load().cbq_quantize_act(_dev_ptr(x2, torch.float32, "x"), K, n, _dev_ptr(qx, torch.int8, "qx"),
                                   _dev_ptr(dx, torch.float32, "dx"), _stream(stream)), "cbq_quantize_act")
    return qx, dx


def _y_out(y, n, M, device):
    torch = _torch()
    if y is None:
        y = torch.empty((n, M), dtype=torch.float32, device=device)
    return y


def cbq_matvec_q(W: Weights, qx, dx, y=None, stream=None):
    torch = _torch()
    n = qx.reshape(-1, W.K).shape[0]
    y = _y_out(y, n, W.M, qx.device)
    _check(load().cbq_matvec_q(W.handle, _dev_ptr(qx, torch.int8, "qx"), _dev_ptr(dx, torch.float32, "dx"), n,
                               _dev_ptr(y, torch.float32, "y"), _stream(stream)), "cbq_matvec_q")
    return y


def cbq_matvec(W: Weights, x, y=None, stream=None):
    torch = _torch()
    n = x.reshape(-1, W.K).shape[0]
    y = _y_out(y, n, W.M, x.device)
    _check(load().cbq_matvec(W.handle, _dev_ptr(x, torch.float32, "x"), n, _dev_ptr(y, torch.float32, "y"),
                             _stream(stream)), "cbq_matvec")
    return y


def cbq_matvec_static(W: Weights, x, y=None, stream=None):
    """cbq_matvec without touching the handle's workspace: the quantized
    activations go to the library's static per-device scratch (no device
    memory is allocated by this call)."""
    torch = _torch()
    n = x.reshape(-1, W.K).shape[0]
    y = _y_out(y, n, W.M, x.device)
    _check(load().cbq_matvec_static(W.handle, _dev_ptr(x, torch.float32, "x"), n, _dev_ptr(y, torch.float32, "y"),
                                    _stream(stream)), "cbq_matvec_static")
    return y


def cbq_matvec_host(W: Weights, x: np.ndarray, y: np.ndarray | None = None, stream=None):
    n = x.reshape(-1, W.K).shape[0]
    if y is None:
        y = np.empty((n, W.M), dtype=np.float32)
    _check(load().cbq_matvec_host(W.handle, _host_ptr(x, np.float32, "x"), n, _host_ptr(y, np.float32, "y"),
                                  _stream(stream)), "cbq_matvec_host")
    return y


def cbq_moe_matvec(L: Moe, h, ids, wts, swiglu: int = 1, y=None, stream=None):
    torch = _torch()
    n_tok, k = ids.shape
    if y is None:
        y = torch.empty((n_tok, L.H), dtype=torch.float32, device=h.device)
    _check(load().cbq_moe_matvec(L.handle, _dev_ptr(h, torch.float32, "h"), n_tok, _dev_ptr(ids, torch.int32, "ids"),
                                 _dev_ptr(wts, torch.float32, "wts"), k, int(swiglu),
                                 _dev_ptr(y, torch.float32, "y"), _stream(stream)), "cbq_moe_matvec")
    return y


def cbq_moe_set_shared(L: Moe, gate_up, down, stream=None):
    """Give L a shared expert (canonical blocks, host array or device tensor),
    or remove it with gate_up = down = None."""
    L.set_shared(gate_up, down, stream=stream)


def cbq_router_topk(logits, k: int, ids=None, wts=None, stream=None):
    """ids (n_tok, k) int32 and fp32 softmax weights of the k largest logits
    of each row of logits (n_tok, E) fp32, on the device."""
    torch = _torch()
    n_tok, E = logits.shape
    if ids is None:
        ids = torch.empty((n_tok, k), dtype=torch.int32, device=logits.device)
    if wts is None:
        wts = torch.empty((n_tok, k), dtype=torch.float32, device=logits.device)
    _check(load().cbq_router_topk(_dev_ptr(logits, torch.float32, "logits"), n_tok, E, k,
                                  _dev_ptr(ids, torch.int32, "ids"), _dev_ptr(wts, torch.float32, "wts"),
                                  _stream(stream)), "cbq_router_topk")
    return ids, wts


def cbq_moe_matvec_logits(L: Moe, h, logits, k: int, swiglu: int = 1, y=None, stream=None):
    """The routed layer from router logits (n_tok, E): top-k selection and
    softmax weights on the device, then cbq_moe_matvec."""
    torch = _torch()
    n_tok = logits.shape[0]
    if y is None:
        y = torch.empty((n_tok, L.H), dtype=torch.float32, device=h.device)
    _check(load().cbq_moe_matvec_logits(L.handle, _dev_ptr(h, torch.float32, "h"), n_tok,
                                        _dev_ptr(logits, torch.float32, "logits"), k, int(swiglu),
                                        _dev_ptr(y, torch.float32, "y"), _stream(stream)), "cbq_moe_matvec_logits")
    return y


def cbq_moe_matvec_host(L: Moe, h: np.ndarray, ids: np.ndarray, wts: np.ndarray, swiglu: int = 1,
                        y: np.ndarray | None = None, stream=None):
    n_tok, k = ids.shape
    if y is None:
        y = np.empty((n_tok, L.H), dtype=np.float32)
    _check(load().cbq_moe_matvec_host(L.handle, _host_ptr(h, np.float32, "h"), n_tok,
                                      _host_ptr(ids, np.int32, "ids"), _host_ptr(wts, np.float32, "wts"), k,
                                      int(swiglu), _host_ptr(y, np.float32, "y"), _stream(stream)),
           "cbq_moe_matvec_host")
    return y


def cbq_weights_get_error(W: Weights, stream=None) -> int:
    """Read and clear W's error word (CBQ_DEVERR_* bits) in the order of the
    stream (default: torch's current stream), then wait for that stream."""
    code = ctypes.c_uint()
    _check(load().cbq_weights_get_error(W.handle, _stream(stream), ctypes.byref(code)), "cbq_weights_get_error")
    return code.value


def cbq_moe_get_error(L: Moe, stream=None) -> int:
    """Read and clear L's error word (CBQ_DEVERR_* bits) in stream order."""
    code = ctypes.c_uint()
    _check(load().cbq_moe_get_error(L.handle, _stream(stream), ctypes.byref(code)), "cbq_moe_get_error")
    return code.value


def cbq_moe_debug_stall(L: Moe, mode: int):
    """Give-up test mode of the layer kernel (0 off; 1 a dependency never met;
    2 a weight stage never filled)."""
    _check(load().cbq_moe_debug_stall(L.handle, int(mode)), "cbq_moe_debug_stall")


def cbq_debug_mmq_stall(W: Weights, mode: int):
    """Give-up test mode of the tensor-core path (0 off; 1 the first CTA
    copies nothing, so its waits run out)."""
    _check(load().cbq_debug_mmq_stall(W.handle, int(mode)), "cbq_debug_mmq_stall")


def cbq_debug_tree_stall(mode: int):
    """Give-up test mode of this thread's cbq_tree_attention calls (0 off; 1
    the many-row kernel's first block copies nothing, so its waits run out)."""
    _check(load().cbq_debug_tree_stall(int(mode)), "cbq_debug_tree_stall")


def cbq_debug_block_dots(W: Weights, qx, s=None, stream=None):
    torch = _torch()
    n = qx.reshape(-1, W.K).shape[0]
    if s is None:
        s = torch.empty((n, W.M, W.K // CBQ_QK), dtype=torch.int32, device=qx.device)
    _check(load().cbq_debug_block_dots(W.handle, _dev_ptr(qx, torch.int8, "qx"), n, _dev_ptr(s, torch.int32, "s"),
                                       _stream(stream)), "cbq_debug_block_dots")
    return s


def cbq_moe_debug_block_dots(L: Moe, e: int, which: int, qx, s=None, stream=None):
    torch = _torch()
    M, K = (2 * L.F, L.H) if which == 0 else (L.H, L.F)
    n = qx.reshape(-1, K).shape[0]
    if s is None:
        s = torch.empty((n, M, K // CBQ_QK), dtype=torch.int32, device=qx.device)
    _check(load().cbq_moe_debug_block_dots(L.handle, e, which, _dev_ptr(qx, torch.int8, "qx"), n,
                                           _dev_ptr(s, torch.int32, "s"), _stream(stream)), "cbq_moe_debug_block_dots")
    return s


def cbq_moe_set_debug(L: Moe, keep: bool):
    _check(load().cbq_moe_set_debug(L.handle, int(bool(keep))), "cbq_moe_set_debug")


def cbq_moe_set_stage_events(L: Moe, events=None):
    """events: three torch.cuda.Event(enable_timing=True) or None to stop."""
    ptrs = [None] * 3 if events is None else [ctypes.c_void_p(ev.cuda_event) for ev in events]
    _check(load().cbq_moe_set_stage_events(L.handle, *ptrs), "cbq_moe_set_stage_events")


def cbq_moe_debug_intermediate(L: Moe, nslots: int, stream=None):
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device())
    a = torch.empty((nslots, L.F), dtype=torch.float32, device=dev)
    qa = torch.empty((nslots, L.F), dtype=torch.int8, device=dev)
    da = torch.empty((nslots, L.F // CBQ_QK), dtype=torch.float32, device=dev)
    _check(load().cbq_moe_debug_intermediate(L.handle, nslots, _dev_ptr(a, torch.float32, "a"),
                                             _dev_ptr(qa, torch.int8, "qa"), _dev_ptr(da, torch.float32, "da"),
                                             _stream(stream)), "cbq_moe_debug_intermediate")
    return a, qa, da


def cbq_quantize_weights(w, out=None, stream=None):
    """Canonical blocks (M, K/32, 18) uint8 of the fp32 matrix w (M, K), both
    on the device (the weight converter)."""
    torch = _torch()
    M, K = w.shape
    if out is None:
        out = torch.empty((M, K // CBQ_QK, CBQ_BLOCK_BYTES), dtype=torch.uint8, device=w.device)
    if not out.is_contiguous() or out.dtype != torch.uint8 or out.numel() != M * (K // CBQ_QK) * CBQ_BLOCK_BYTES:
        raise ValueError("out must be a contiguous uint8 tensor of M x K/32 x 18 bytes")
    _check(load().cbq_quantize_weights(_dev_ptr(w, torch.float32, "w"), M, K, ctypes.c_void_p(out.data_ptr()),
                                       _stream(stream)), "cbq_quantize_weights")
    return out


def cbq_hc_sinkhorn(logits, iters, out=None, stream=None):
    """Sinkhorn normalisation of the fp32 hyper-connection logits (..., 4, 4)
    on the device: exp(c - max c), then `iters` rounds of row and column
    normalisation; out (same shape) may be logits itself."""
    torch = _torch()
    if logits.dim() < 2 or tuple(logits.shape[-2:]) != (CBQ_HC_NHC, CBQ_HC_NHC):
        raise ValueError(f"logits must end in ({CBQ_HC_NHC}, {CBQ_HC_NHC})")
    if out is None:
        out = torch.empty_like(logits)
    if out.shape != logits.shape:
        raise ValueError("out must have the shape of logits")
    n = logits.numel() // (CBQ_HC_NHC * CBQ_HC_NHC)
    _check(load().cbq_hc_sinkhorn(_dev_ptr(logits, torch.float32, "logits"), n, int(iters),
                                  _dev_ptr(out, torch.float32, "out"), _stream(stream)), "cbq_hc_sinkhorn")
    return out


def cbq_matmat(W: Weights, x, y=None, stream=None):
    """y (n, M) fp32 = W applied to the n <= 16 fp32 columns x (n, K), by the
    tensor-core path; x and y on the device."""
    torch = _torch()
    n = x.shape[0]
    if y is None:
        y = torch.empty((n, W.M), dtype=torch.float32, device=x.device)
    _check(load().cbq_matmat(W.handle, _dev_ptr(x, torch.float32, "x"), n, _dev_ptr(y, torch.float32, "y"),
                             _stream(stream)), "cbq_matmat")
    return y


def cbq_debug_mmq_block_dots(W: Weights, qx, stream=None):
    """The exact block dots (n, M, K/32) int32 of W with int8 columns qx (n, K), by the tensor-core path."""
    torch = _torch()
    n = qx.shape[0]
    s = torch.empty((n, W.M, W.K // CBQ_QK), dtype=torch.int32, device=qx.device)
    _check(load().cbq_debug_mmq_block_dots(W.handle, _dev_ptr(qx, torch.int8, "qx"), n,
                                           _dev_ptr(s, torch.int32, "s"), _stream(stream)), "cbq_debug_mmq_block_dots")
    return s


# ------------------------------------- positions, attention, sampling --
#
# A small call of these takes the GPU about as long as Python takes to make
# it, so the marshalling looks each tensor property up once and calls into
# torch only where it has to.

_SCALINGS = {"none": CBQ_ROPE_NONE, "linear": CBQ_ROPE_LINEAR, "turns": CBQ_ROPE_BY_TURNS, "index": CBQ_ROPE_BY_INDEX}
_LAYOUTS = {"half": CBQ_ROPE_HALF, "pairs": CBQ_ROPE_PAIRS}


@functools.cache
def _codes():
    torch = _torch()
    return {torch.float32: CBQ_F32, torch.bfloat16: CBQ_BF16, torch.float16: CBQ_F16}


def _dtype(t, name):
    code = _codes().get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _raw_stream(stream, t):
    """The cudaStream_t of `stream`, or of torch's current one on t's device."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


def _new(shape, dtype, device, stream, returned=True):
    """A new tensor that kernels on `stream` (None: torch's current one) write.

    Torch orders a block only with the stream it was taken for: one of the
    current stream's may still be in use there when `stream` writes it, and one
    that is dropped goes to the current stream's next allocation while `stream`
    still works on it.  So it is taken for `stream`; what the caller gets is
    marked as used on the current stream too, where the caller goes on with it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _layout(layout):
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    return code


def _heads(t, name):
    """(pointer, token stride, head stride) of a CUDA tensor (tokens, heads,
    dim) whose last axis is contiguous."""
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] != 1):
        raise ValueError(f"{name} must be (tokens, heads, dim) with a contiguous last axis")
    return t.data_ptr(), st[0], st[1]


def _cache(kc, vc):
    """cbq_kv_cache of two CUDA tensors (pages, page_size, kv_heads, dim)."""
    if not kc.is_cuda or not vc.is_cuda or kc.dtype != vc.dtype:
        raise TypeError("kc and vc must be CUDA tensors of one dtype")
    shape, st = kc.shape, kc.stride()
    if len(shape) != 4 or shape != vc.shape or st != vc.stride():
        raise ValueError("kc and vc must be (pages, page_size, kv_heads, dim) of one shape and strides")
    pages, page, heads, dim = shape
    if st[3] != 1 and dim != 1:
        raise ValueError("the cache's last axis must be contiguous")
    return cbq_kv_cache(kc.data_ptr(), vc.data_ptr(), _dtype(kc, "kc"), heads, dim, page, pages, st[0], st[1], st[2])


def _vec(t, dtype, n, name):
    """Pointer of a contiguous CUDA tensor of n values of dtype (n < 0: any number)."""
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if not t.is_contiguous() or (n >= 0 and t.numel() != n):
        raise ValueError(f"{name} must be contiguous" + (f" with {n} values" if n >= 0 else ""))
    return t.data_ptr()


def _opt_vec(t, dtype, n, name):
    return None if t is None else _vec(t, dtype, n, name)


def cbq_rope_turns(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                   orig_len: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """The fp64 table of a rotation (rot_dim/2 turns a position) on `device`
    (default: the current CUDA device); scaling "none", "linear", "turns" or
    "index"."""
    torch = _torch()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    t = np.empty(max(int(rot_dim) // 2, 1), dtype=np.float64)
    _check(load().cbq_rope_turns(int(rot_dim), base, _SCALINGS[scaling], factor, orig_len, low, high,
                                 t.ctypes.data_as(_P)), "cbq_rope_turns")
    return torch.from_numpy(t).to("cuda" if device is None else device)


def cbq_rope(x, pos, turns, rot_off: int = 0, layout: str = "half", mscale: float = 1.0, out=None, stream=None):
    """Rotary positions of x (tokens, heads, dim): 2 * len(turns) values of
    each head from rot_off on turn, the others are copied; pos (tokens) int32,
    turns fp64 (cbq_rope_turns).  out may be x."""
    torch = _torch()
    n, heads, dim = x.shape
    xp, xt, xh = _heads(x, "x")
    if out is None:
        out = _new((n, heads, dim), x.dtype, x.device, stream)
        op, ot, oh = out.data_ptr(), heads * dim, dim
    else:
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have the shape and dtype of x")
        op, ot, oh = _heads(out, "out")
    _check(load().cbq_rope(xp, _dtype(x, "x"), n, heads, dim, xt, xh, _vec(pos, torch.int32, n, "pos"),
                           _vec(turns, torch.float64, -1, "turns"), 2 * turns.numel(), rot_off, _layout(layout),
                           mscale, op, ot, oh, _raw_stream(stream, x)), "cbq_rope")
    return out


def cbq_rope_append(q, k, v, pos, slots, turns, kc, vc, rot_off: int = 0, layout: str = "half", mscale: float = 1.0,
                    out=None, err=None, stream=None):
    """New tokens' q (tokens, q_heads, dim) rotated (returned, in the cache's
    dtype), their k rotated and v copied into the paged cache kc, vc (pages,
    page_size, kv_heads, dim) at slots (tokens) int64 (negative: not written).
    err: an optional int32 tensor of one value for the CBQ_DEVERR_* bits."""
    torch = _torch()
    shape = q.shape
    n, heads, dim = shape
    c = _cache(kc, vc)
    if k.shape != (n, c.kv_heads, dim) or v.shape != k.shape or dim != c.head_dim:
        raise ValueError("k and v must be (tokens, kv_heads, dim) as the cache, dim as q")
    qp, qt, qh = _heads(q, "q")
    kp, kt, kh = _heads(k, "k")
    vp, vt, vh = _heads(v, "v")
    if kt != vt or kh != vh or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype, and k and v one set of strides")
    if out is None:
        out = _new(shape, kc.dtype, q.device, stream)
        op = out.data_ptr()
    else:
        op = _vec(out, kc.dtype, n * heads * dim, "out")
    _check(load().cbq_rope_append(qp, kp, vp, _dtype(q, "q"), n, heads, qt, qh, kt, kh,
                                  _vec(pos, torch.int32, n, "pos"), _vec(slots, torch.int64, n, "slots"),
                                  _vec(turns, torch.float64, -1, "turns"), 2 * turns.numel(), rot_off,
                                  _layout(layout), mscale, c, op,
                                  _opt_vec(err, torch.int32, 1, "err"), _raw_stream(stream, q)), "cbq_rope_append")
    return out


@functools.lru_cache(1024)
def cbq_tree_attention_workspace(n_seq: int, total_tok: int, max_tok: int, max_len: int, q_heads: int, kv_heads: int,
                                 head_dim: int) -> int:
    """Bytes of workspace of cbq_tree_attention for these limits."""
    b = ctypes.c_int64()
    _check(load().cbq_tree_attention_workspace(n_seq, total_tok, max_tok, max_len, q_heads, kv_heads, head_dim,
                                               ctypes.byref(b)), "cbq_tree_attention_workspace")
    return b.value


@functools.cache
def _least_workspace(dev):
    """What calls that need no workspace pass for one (nothing is written there)."""
    return _torch().empty(16, dtype=_torch().uint8, device=dev)


def cbq_tree_attention(q, kc, vc, table, ctx, start, mask, max_tok: int, max_len: int, scale: float | None = None,
                       out=None, with_lse: bool = False, workspace=None, err=None, stream=None):
    """Attention of each sequence's drafted tokens, packed in q (tokens,
    q_heads, dim), over its committed tokens and those drafts its mask names,
    in the paged cache kc, vc: table (sequences, width) int32 page ids, ctx
    (sequences) int32 committed lengths, start (sequences + 1) int32 first rows,
    mask (tokens) int64 bits.  scale: dim ** -0.5 if None.  Returns out, or
    (out, lse) with with_lse.  workspace: a uint8 tensor of
    cbq_tree_attention_workspace bytes (allocated when None)."""
    torch = _torch()
    shape, dev, i32 = q.shape, q.device, torch.int32
    n, heads, dim = shape
    c = _cache(kc, vc)
    if q.dtype != kc.dtype or dim != c.head_dim:
        raise ValueError("q must have the cache's dtype and dim")
    n_seq, width = table.shape
    if out is None:
        out = _new(shape, q.dtype, dev, stream)
        op, od = out.data_ptr(), c.dtype
    else:
        if out.shape != shape:
            raise ValueError("out must have the shape of q")
        op, od = _vec(out, out.dtype, n * heads * dim, "out"), _dtype(out, "out")
    lse = _new((n, heads), torch.float32, dev, stream) if with_lse else None
    if workspace is None:
        room = cbq_tree_attention_workspace(n_seq, n, max_tok, max_len, heads, c.kv_heads, dim)
        workspace = _least_workspace(dev) if room <= 16 else _new((room,), torch.uint8, dev, stream, returned=False)
        wp = workspace.data_ptr()
    else:
        wp, room = _vec(workspace, torch.uint8, -1, "workspace"), workspace.numel()
    qp, qt, qh = _heads(q, "q")
    _check(load().cbq_tree_attention(qp, qt, qh, heads, n, c, _vec(table, i32, -1, "table"), width, n_seq,
                                     _vec(ctx, i32, n_seq, "ctx"), _vec(start, i32, n_seq + 1, "start"),
                                     _vec(mask, torch.int64, n, "mask"), max_tok, max_len,
                                     dim ** -0.5 if scale is None else scale,
                                     op, od, None if lse is None else lse.data_ptr(), wp, room,
                                     _opt_vec(err, i32, 1, "err"), _raw_stream(stream, q)), "cbq_tree_attention")
    return (out, lse) if with_lse else out


def cbq_sample(logits, temperature, top_k, top_p, min_p, u, ids=None, probs=None, stream=None):
    """One token from each row of logits (rows, V): temperature, top_p, min_p
    and u (rows) fp32, top_k (rows) int32, each but u may be None.  Returns
    ids int32 and the drawn tokens' probabilities among the kept ones."""
    torch = _torch()
    n, V = logits.shape
    st = logits.stride()
    if not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    if st[1] != 1 and V != 1:
        raise ValueError("logits must have a contiguous last axis")
    f, i32 = torch.float32, torch.int32
    if ids is None:
        ids = _new((n,), i32, logits.device, stream)
        ip = ids.data_ptr()
    else:
        ip = _vec(ids, i32, n, "ids")
    if probs is None:
        probs = _new((n,), f, logits.device, stream)
        pp = probs.data_ptr()
    else:
        pp = _vec(probs, f, n, "probs")
    _check(load().cbq_sample(logits.data_ptr(), _dtype(logits, "logits"), n, V, st[0],
                             _opt_vec(temperature, f, n, "temperature"), _opt_vec(top_k, i32, n, "top_k"),
                             _opt_vec(top_p, f, n, "top_p"), _opt_vec(min_p, f, n, "min_p"), _vec(u, f, n, "u"),
                             ip, pp, _raw_stream(stream, logits)),
           "cbq_sample")
    return ids, probs
