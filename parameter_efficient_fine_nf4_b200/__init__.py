"""Python binding of libqlora (the QLoRA linear layer on B200).

Argument marshalling only: every step runs in the CUDA kernels of
``libqlora.so``, reached through its C ABI (``include/qlora.h``).  PyTorch
provides device memory and the current stream.  If the shared library is
missing the import of any call raises; there is no CPU fallback.

Names mirror the C entry points.  bf16 tensors are ``torch.bfloat16``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

QLORA_OK = 0
QLORA_ERR_TIMEOUT = 6
BLOCK = 64
BLOCK2 = 256


class QloraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


class _NF4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("scale2", ctypes.c_void_p), ("mean", ctypes.c_void_p),
                ("d", ctypes.c_int64), ("k", ctypes.c_int64),
                ("block", ctypes.c_int32), ("block2", ctypes.c_int32)]


class _Pool(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("Bt", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("k", ctypes.c_int64), ("d", ctypes.c_int64), ("n", ctypes.c_int32), ("width", ctypes.c_int32)]


class _Requests(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("order", ctypes.c_void_p),
                ("seg", ctypes.c_void_p), ("tile_first", ctypes.c_void_p), ("tiles", ctypes.c_void_p),
                ("T", ctypes.c_int64), ("n_req", ctypes.c_int32), ("n", ctypes.c_int32)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


_lib = None

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIZE = ctypes.c_size_t
_INT = ctypes.c_int
_F = ctypes.c_float
_NF4P = ctypes.POINTER(_NF4)
_POOLP = ctypes.POINTER(_Pool)
_REQP = ctypes.POINTER(_Requests)

_SIGNATURES = {
    "qlora_strerror": (ctypes.c_char_p, [_INT]),
    "qlora_version": (_INT, []),
    "qlora_nf4_levels": (_INT, [_VP, _VP]),
    "qlora_quantize_workspace_bytes": (_SIZE, [_I64, _I64]),
    "qlora_nf4_quantize": (_INT, [_VP, _I64, _I64, _INT, _NF4P, _VP, _SIZE, _VP]),
    "qlora_nf4_dequantize": (_INT, [_NF4P, _VP, _VP]),
    "qlora_nf4_quantize_noalloc": (_INT, [_VP, _I64, _I64, _INT, _NF4P, _VP]),
    "qlora_fwd_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "qlora_fwd": (_INT, [_NF4P, _VP, _VP, _INT, _F, _VP, _I64, _VP, _VP, _VP, _SIZE, _VP]),
    "qlora_bwd_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "qlora_bwd": (_INT, [_NF4P, _VP, _VP, _INT, _F, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _VP,
                         _SIZE, _VP]),
    "qlora_fwd_dropout_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "qlora_fwd_dropout": (_INT, [_NF4P, _VP, _VP, _INT, _F, _VP, _VP, _F, _I64, _VP, _VP, _VP, _SIZE, _VP]),
    "qlora_bwd_dropout_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "qlora_bwd_dropout": (_INT, [_NF4P, _VP, _VP, _INT, _F, _VP, _VP, _F, _VP, _VP, _I64, _VP, _VP, _VP, _VP,
                                 _SIZE, _VP]),
    "qlora_fwd_multi_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _INT, _I64]),
    "qlora_fwd_multi": (_INT, [_NF4P, _INT, _VP, _VP, _INT, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _SIZE, _VP]),
    "qlora_bwd_multi_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _INT, _I64]),
    "qlora_bwd_multi": (_INT, [_NF4P, _INT, _VP, _VP, _INT, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _VP,
                               _SIZE, _VP]),
    "lora_fwd_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "lora_fwd": (_INT, [_VP, _I64, _I64, _VP, _VP, _INT, _F, _VP, _I64, _VP, _VP, _VP, _SIZE, _VP]),
    "lora_bwd_workspace_bytes": (_SIZE, [_I64, _I64, _INT, _I64]),
    "lora_bwd": (_INT, [_VP, _I64, _I64, _VP, _VP, _INT, _F, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _VP,
                        _SIZE, _VP]),
    "lora_adam_step": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _F, _F, _F, _F, _F, _VP]),
    "lora_requests_max_tiles": (_I64, [_INT, _INT, _I64]),
    "lora_requests_plan": (_INT, [_VP, _VP, _REQP, _VP]),
    "lora_requests_fwd_workspace_bytes": (_SIZE, [_POOLP, _REQP]),
    "lora_requests_fwd": (_INT, [_POOLP, _REQP, _VP, _VP, _VP, _VP, _VP, _SIZE, _VP]),
    "lora_requests_bwd_workspace_bytes": (_SIZE, [_POOLP, _REQP]),
    "lora_requests_bwd": (_INT, [_POOLP, _REQP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SIZE, _VP]),
    "qlora_fwd_requests_workspace_bytes": (_SIZE, [_NF4P, _POOLP, _REQP]),
    "qlora_fwd_requests": (_INT, [_NF4P, _POOLP, _REQP, _VP, _VP, _VP, _VP, _SIZE, _VP]),
    "qlora_bwd_requests_workspace_bytes": (_SIZE, [_NF4P, _POOLP, _REQP]),
    "qlora_bwd_requests": (_INT, [_NF4P, _POOLP, _REQP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SIZE, _VP]),
    "lora_muon_workspace_bytes": (_SIZE, [_I64, _I64, _I64]),
    "lora_muon_step": (_INT, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _F, _F, _INT, _F, _F, _F, _INT, _VP, _VP, _SIZE,
                              _VP]),
    "lora_merge_workspace_bytes": (_SIZE, [_I64, _I64, _INT]),
    "lora_merge": (_INT, [_NF4P, _VP, _VP, _INT, _F, _VP, _VP, _SIZE, _VP]),
    "lora_unmerge": (_INT, [_VP, _VP, _VP, _INT, _F, _I64, _I64, _VP, _VP, _SIZE, _VP]),
    "qlora_get_device_status": (_INT, [_VP, ctypes.POINTER(_INT)]),
    "qlora_selftest_wait_timeout": (_INT, [_INT, _VP]),
    "qlora_profile_begin": (_INT, []),
    "qlora_profile_end": (_INT, [ctypes.POINTER(KernelStat), _INT, ctypes.POINTER(_INT)]),
    "qlora_launch_count": (_I64, []),
    "qlora_set_nf4_gemm_mode": (_INT, [_INT]),
    "qlora_comm_unique_id": (_INT, [_VP]),
    "qlora_comm_init": (_INT, [_VP, _INT, _INT, ctypes.POINTER(_VP)]),
    "qlora_comm_destroy": (_INT, [_VP]),
    "qlora_grad_allreduce": (_INT, [_VP, _VP, _I64, _VP, _I64, _VP]),
}

EXPORTED = tuple(_SIGNATURES)


def lib() -> ctypes.CDLL:
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libqlora.so not found at {LIB_PATH}; build it with "
                "`python -m parameter_efficient_fine_nf4_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().qlora_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != QLORA_OK:
        raise QloraError(status, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libqlora must be contiguous")
    return t.data_ptr()


def _need(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")


class NF4Weight:
    """Device buffers of one NF4 + double-quant weight (the qlora_nf4_t)."""

    def __init__(self, d: int, k: int, device=None):
        device = torch.device("cuda") if device is None else torch.device(device)
        n_b = d * k // BLOCK
        n_g = (n_b + BLOCK2 - 1) // BLOCK2
        self.d, self.k = d, k
        self.codes = torch.empty(d * k // 2, dtype=torch.uint8, device=device)
        self.absmax_q = torch.empty(n_b, dtype=torch.uint8, device=device)
        self.scale2 = torch.empty(n_g, dtype=torch.float32, device=device)
        self.mean = torch.empty(1, dtype=torch.float32, device=device)
        self._c = _NF4(self.codes.data_ptr(), self.absmax_q.data_ptr(), self.scale2.data_ptr(),
                       self.mean.data_ptr(), d, k, BLOCK, BLOCK2)

    @property
    def cstruct(self) -> _NF4:
        return self._c

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.absmax_q, self.scale2, self.mean))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    device = torch.device("cuda") if device is None else torch.device(device)
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------- host-only
def qlora_version() -> int:
    return lib().qlora_version()


def qlora_nf4_levels():
    lv = (ctypes.c_float * 16)()
    th = (ctypes.c_float * 15)()
    _check(lib().qlora_nf4_levels(ctypes.addressof(lv), ctypes.addressof(th)), "qlora_nf4_levels")
    return list(lv), list(th)


def qlora_quantize_workspace_bytes(d: int, k: int) -> int:
    return lib().qlora_quantize_workspace_bytes(d, k)


def qlora_fwd_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().qlora_fwd_workspace_bytes(d, k, r, T)


def qlora_bwd_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().qlora_bwd_workspace_bytes(d, k, r, T)


def lora_merge_workspace_bytes(d: int, k: int, r: int) -> int:
    return lib().lora_merge_workspace_bytes(d, k, r)


def qlora_launch_count() -> int:
    return lib().qlora_launch_count()


def qlora_set_nf4_gemm_mode(mode: int) -> None:
    """0 = by shape, 1 = one CTA per tile, 2 = CTA pairs (same bits, other speed)."""
    _check(lib().qlora_set_nf4_gemm_mode(mode), "qlora_set_nf4_gemm_mode")


# ------------------------------------------------------------------- device calls
def qlora_nf4_quantize(W0: torch.Tensor, out: Optional[NF4Weight] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> NF4Weight:
    d, k = W0.shape
    _need(W0, torch.float32, (d, k), "W0")
    out = NF4Weight(d, k, W0.device) if out is None else out
    nbytes = qlora_quantize_workspace_bytes(d, k)
    ws = workspace(nbytes, W0.device) if ws is None else ws
    st = lib().qlora_nf4_quantize(_ptr(W0), d, k, BLOCK, ctypes.byref(out.cstruct), _ptr(ws),
                                  ws.numel(), _stream(stream))
    _check(st, "qlora_nf4_quantize")
    return out


NOALLOC_MAX_WEIGHTS = 1 << 28


def qlora_nf4_quantize_noalloc(W0: torch.Tensor, out: NF4Weight, stream=None) -> NF4Weight:
    """Quantise using the library's static device scratch (no workspace).

    For callers that cannot allocate device memory: pass preallocated output
    buffers in ``out``; nothing else is allocated.  d*k is limited to 2^28.
    Calls share one scratch array, so calls that overlap on the GPU race.
    """
    d, k = W0.shape
    _need(W0, torch.float32, (d, k), "W0")
    st = lib().qlora_nf4_quantize_noalloc(_ptr(W0), d, k, BLOCK, ctypes.byref(out.cstruct),
                                          _stream(stream))
    _check(st, "qlora_nf4_quantize_noalloc")
    return out


def qlora_nf4_dequantize(q: NF4Weight, W_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    W_out = torch.empty(q.d, q.k, dtype=torch.bfloat16, device=q.codes.device) if W_out is None else W_out
    _need(W_out, torch.bfloat16, (q.d, q.k), "W_out")
    _check(lib().qlora_nf4_dequantize(ctypes.byref(q.cstruct), _ptr(W_out), _stream(stream)),
           "qlora_nf4_dequantize")
    return W_out


def qlora_fwd(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
              Y: Optional[torch.Tensor] = None, U_save: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    r = A.shape[0]
    T = X.shape[0]
    _need(A, torch.bfloat16, (r, q.k), "A")
    _need(B, torch.bfloat16, (q.d, r), "B")
    _need(X, torch.bfloat16, (T, q.k), "X")
    dev = X.device
    Y = torch.empty(T, q.d, dtype=torch.bfloat16, device=dev) if Y is None else Y
    U_save = torch.empty(T, r, dtype=torch.float32, device=dev) if U_save is None else U_save
    _need(Y, torch.bfloat16, (T, q.d), "Y")
    _need(U_save, torch.float32, (T, r), "U_save")
    nbytes = qlora_fwd_workspace_bytes(q.d, q.k, r, T)
    ws = workspace(nbytes, dev) if ws is None else ws
    st = lib().qlora_fwd(ctypes.byref(q.cstruct), _ptr(A), _ptr(B), r, float(alpha), _ptr(X), T,
                         _ptr(Y), _ptr(U_save), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qlora_fwd")
    return Y, U_save


def qlora_bwd(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
              U_saved: torch.Tensor, dY: torch.Tensor, dX: Optional[torch.Tensor] = None,
              dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None):
    r = A.shape[0]
    T = X.shape[0]
    _need(A, torch.bfloat16, (r, q.k), "A")
    _need(B, torch.bfloat16, (q.d, r), "B")
    _need(X, torch.bfloat16, (T, q.k), "X")
    _need(U_saved, torch.float32, (T, r), "U_saved")
    _need(dY, torch.bfloat16, (T, q.d), "dY")
    dev = X.device
    dX = torch.empty(T, q.k, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dA = torch.empty(r, q.k, dtype=torch.float32, device=dev) if dA is None else dA
    dB = torch.empty(q.d, r, dtype=torch.float32, device=dev) if dB is None else dB
    _need(dX, torch.bfloat16, (T, q.k), "dX")
    _need(dA, torch.float32, (r, q.k), "dA")
    _need(dB, torch.float32, (q.d, r), "dB")
    nbytes = qlora_bwd_workspace_bytes(q.d, q.k, r, T)
    ws = workspace(nbytes, dev) if ws is None else ws
    st = lib().qlora_bwd(ctypes.byref(q.cstruct), _ptr(A), _ptr(B), r, float(alpha), _ptr(X),
                         _ptr(U_saved), _ptr(dY), T, _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                         ws.numel(), _stream(stream))
    _check(st, "qlora_bwd")
    return dX, dA, dB


def qlora_fwd_dropout_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().qlora_fwd_dropout_workspace_bytes(d, k, r, T)


def qlora_bwd_dropout_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().qlora_bwd_dropout_workspace_bytes(d, k, r, T)


def _need_keep(keep: Optional[torch.Tensor], T: int, k: int, p: float):
    if p == 0.0 and keep is None:
        return None
    _need(keep, torch.uint8, (T * k // 8,), "keep")
    return _ptr(keep)


def qlora_fwd_dropout(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
                      keep: Optional[torch.Tensor], p: float, Y: Optional[torch.Tensor] = None,
                      U_save: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Forward with LoRA dropout on the adapter input (keep: bit-packed T*k/8 bytes)."""
    r = A.shape[0]
    T = X.shape[0]
    _need(A, torch.bfloat16, (r, q.k), "A")
    _need(B, torch.bfloat16, (q.d, r), "B")
    _need(X, torch.bfloat16, (T, q.k), "X")
    kp = _need_keep(keep, T, q.k, p)
    dev = X.device
    Y = torch.empty(T, q.d, dtype=torch.bfloat16, device=dev) if Y is None else Y
    U_save = torch.empty(T, r, dtype=torch.float32, device=dev) if U_save is None else U_save
    _need(Y, torch.bfloat16, (T, q.d), "Y")
    _need(U_save, torch.float32, (T, r), "U_save")
    ws = workspace(qlora_fwd_dropout_workspace_bytes(q.d, q.k, r, T), dev) if ws is None else ws
    st = lib().qlora_fwd_dropout(ctypes.byref(q.cstruct), _ptr(A), _ptr(B), r, float(alpha), _ptr(X), kp,
                                 float(p), T, _ptr(Y), _ptr(U_save), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qlora_fwd_dropout")
    return Y, U_save


def qlora_bwd_dropout(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
                      keep: Optional[torch.Tensor], p: float, U_saved: torch.Tensor, dY: torch.Tensor,
                      dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                      dB: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of qlora_fwd_dropout with the same keep mask."""
    r = A.shape[0]
    T = X.shape[0]
    _need(A, torch.bfloat16, (r, q.k), "A")
    _need(B, torch.bfloat16, (q.d, r), "B")
    _need(X, torch.bfloat16, (T, q.k), "X")
    _need(U_saved, torch.float32, (T, r), "U_saved")
    _need(dY, torch.bfloat16, (T, q.d), "dY")
    kp = _need_keep(keep, T, q.k, p)
    dev = X.device
    dX = torch.empty(T, q.k, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dA = torch.empty(r, q.k, dtype=torch.float32, device=dev) if dA is None else dA
    dB = torch.empty(q.d, r, dtype=torch.float32, device=dev) if dB is None else dB
    _need(dX, torch.bfloat16, (T, q.k), "dX")
    _need(dA, torch.float32, (r, q.k), "dA")
    _need(dB, torch.float32, (q.d, r), "dB")
    ws = workspace(qlora_bwd_dropout_workspace_bytes(q.d, q.k, r, T), dev) if ws is None else ws
    st = lib().qlora_bwd_dropout(ctypes.byref(q.cstruct), _ptr(A), _ptr(B), r, float(alpha), _ptr(X), kp,
                                 float(p), _ptr(U_saved), _ptr(dY), T, _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                                 ws.numel(), _stream(stream))
    _check(st, "qlora_bwd_dropout")
    return dX, dA, dB


def _host_alphas(alphas):
    arr = (ctypes.c_float * len(alphas))(*[float(a) for a in alphas])
    return arr


def qlora_fwd_multi(q: NF4Weight, As: torch.Tensor, Bs: torch.Tensor, alphas, idx: torch.Tensor,
                    X: torch.Tensor, Y: Optional[torch.Tensor] = None, U_save: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Forward with a stack of n adapters (As n x r x k, Bs n x d x r), token t
    using adapter idx[t] (int32, device) with scale alphas[idx[t]] / r."""
    n, r = As.shape[0], As.shape[1]
    T = X.shape[0]
    _need(As, torch.bfloat16, (n, r, q.k), "As")
    _need(Bs, torch.bfloat16, (n, q.d, r), "Bs")
    _need(idx, torch.int32, (T,), "idx")
    _need(X, torch.bfloat16, (T, q.k), "X")
    if len(alphas) != n:
        raise ValueError("one alpha per adapter")
    dev = X.device
    Y = torch.empty(T, q.d, dtype=torch.bfloat16, device=dev) if Y is None else Y
    U_save = torch.empty(T, r, dtype=torch.float32, device=dev) if U_save is None else U_save
    _need(Y, torch.bfloat16, (T, q.d), "Y")
    _need(U_save, torch.float32, (T, r), "U_save")
    ws = workspace(lib().qlora_fwd_multi_workspace_bytes(q.d, q.k, n, r, T), dev) if ws is None else ws
    al = _host_alphas(alphas)
    st = lib().qlora_fwd_multi(ctypes.byref(q.cstruct), n, _ptr(As), _ptr(Bs), r, ctypes.addressof(al), _ptr(idx),
                               _ptr(X), T, _ptr(Y), _ptr(U_save), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qlora_fwd_multi")
    return Y, U_save


def qlora_bwd_multi(q: NF4Weight, As: torch.Tensor, Bs: torch.Tensor, alphas, idx: torch.Tensor,
                    X: torch.Tensor, U_saved: torch.Tensor, dY: torch.Tensor, dX: Optional[torch.Tensor] = None,
                    dAs: Optional[torch.Tensor] = None, dBs: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of qlora_fwd_multi: dX and per-adapter dAs (n x r x k), dBs (n x d x r)."""
    n, r = As.shape[0], As.shape[1]
    T = X.shape[0]
    _need(As, torch.bfloat16, (n, r, q.k), "As")
    _need(Bs, torch.bfloat16, (n, q.d, r), "Bs")
    _need(idx, torch.int32, (T,), "idx")
    _need(X, torch.bfloat16, (T, q.k), "X")
    _need(U_saved, torch.float32, (T, r), "U_saved")
    _need(dY, torch.bfloat16, (T, q.d), "dY")
    if len(alphas) != n:
        raise ValueError("one alpha per adapter")
    dev = X.device
    dX = torch.empty(T, q.k, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dAs = torch.empty(n, r, q.k, dtype=torch.float32, device=dev) if dAs is None else dAs
    dBs = torch.empty(n, q.d, r, dtype=torch.float32, device=dev) if dBs is None else dBs
    _need(dX, torch.bfloat16, (T, q.k), "dX")
    _need(dAs, torch.float32, (n, r, q.k), "dAs")
    _need(dBs, torch.float32, (n, q.d, r), "dBs")
    ws = workspace(lib().qlora_bwd_multi_workspace_bytes(q.d, q.k, n, r, T), dev) if ws is None else ws
    al = _host_alphas(alphas)
    st = lib().qlora_bwd_multi(ctypes.byref(q.cstruct), n, _ptr(As), _ptr(Bs), r, ctypes.addressof(al), _ptr(idx),
                               _ptr(X), _ptr(U_saved), _ptr(dY), T, _ptr(dX), _ptr(dAs), _ptr(dBs), _ptr(ws),
                               ws.numel(), _stream(stream))
    _check(st, "qlora_bwd_multi")
    return dX, dAs, dBs


def lora_fwd_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().lora_fwd_workspace_bytes(d, k, r, T)


def lora_bwd_workspace_bytes(d: int, k: int, r: int, T: int) -> int:
    return lib().lora_bwd_workspace_bytes(d, k, r, T)


def lora_fwd(W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
             Y: Optional[torch.Tensor] = None, U_save: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Plain LoRA forward on a bf16 base W (d x k); see lora_fwd in qlora.h."""
    d, k = W.shape
    r = A.shape[0]
    T = X.shape[0]
    _need(W, torch.bfloat16, (d, k), "W")
    _need(A, torch.bfloat16, (r, k), "A")
    _need(B, torch.bfloat16, (d, r), "B")
    _need(X, torch.bfloat16, (T, k), "X")
    dev = X.device
    Y = torch.empty(T, d, dtype=torch.bfloat16, device=dev) if Y is None else Y
    U_save = torch.empty(T, r, dtype=torch.float32, device=dev) if U_save is None else U_save
    _need(Y, torch.bfloat16, (T, d), "Y")
    _need(U_save, torch.float32, (T, r), "U_save")
    ws = workspace(lora_fwd_workspace_bytes(d, k, r, T), dev) if ws is None else ws
    st = lib().lora_fwd(_ptr(W), d, k, _ptr(A), _ptr(B), r, float(alpha), _ptr(X), T, _ptr(Y),
                        _ptr(U_save), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lora_fwd")
    return Y, U_save


def lora_bwd(W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float, X: torch.Tensor,
             U_saved: torch.Tensor, dY: torch.Tensor, dX: Optional[torch.Tensor] = None,
             dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None, stream=None):
    """Plain LoRA backward on a bf16 base W (d x k); see lora_bwd in qlora.h."""
    d, k = W.shape
    r = A.shape[0]
    T = X.shape[0]
    _need(W, torch.bfloat16, (d, k), "W")
    _need(A, torch.bfloat16, (r, k), "A")
    _need(B, torch.bfloat16, (d, r), "B")
    _need(X, torch.bfloat16, (T, k), "X")
    _need(U_saved, torch.float32, (T, r), "U_saved")
    _need(dY, torch.bfloat16, (T, d), "dY")
    dev = X.device
    dX = torch.empty(T, k, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dA = torch.empty(r, k, dtype=torch.float32, device=dev) if dA is None else dA
    dB = torch.empty(d, r, dtype=torch.float32, device=dev) if dB is None else dB
    _need(dX, torch.bfloat16, (T, k), "dX")
    _need(dA, torch.float32, (r, k), "dA")
    _need(dB, torch.float32, (d, r), "dB")
    ws = workspace(lora_bwd_workspace_bytes(d, k, r, T), dev) if ws is None else ws
    st = lib().lora_bwd(_ptr(W), d, k, _ptr(A), _ptr(B), r, float(alpha), _ptr(X), _ptr(U_saved),
                        _ptr(dY), T, _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                        _stream(stream))
    _check(st, "lora_bwd")
    return dX, dA, dB


def lora_adam_step(master: torch.Tensor, weight_bf16: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                   grad: torch.Tensor, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, weight_decay: float = 0.0, stream=None) -> None:
    """One Adam step in place on (master, m, v) and the bf16 copy; see qlora.h."""
    n = master.numel()
    _need(master, torch.float32, tuple(master.shape), "master")
    for t, dt, name in ((weight_bf16, torch.bfloat16, "weight_bf16"), (m, torch.float32, "m"),
                        (v, torch.float32, "v"), (grad, torch.float32, "grad")):
        _need(t, dt, tuple(master.shape), name)
    _check(lib().lora_adam_step(_ptr(master), _ptr(weight_bf16), _ptr(m), _ptr(v), _ptr(grad), n, int(step),
                                float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                                _stream(stream)), "lora_adam_step")


# ------------------------------------------------- many adapters at once (requests)
class _On:
    """The device a call runs on: gives the raw stream, makes the device
    current, allocates on the call's stream (so that a temporary's memory is
    reused in that stream's order) and restores both."""

    __slots__ = ("device", "stream", "held")

    def __init__(self, device, stream):
        self.device, self.stream, self.held = device, stream, None

    def __enter__(self):
        device, stream = self.device, self.stream
        here = device.index == torch._C._cuda_getDevice()
        if stream is None and here:              # the usual call: nothing to switch
            return torch._C._cuda_getCurrentRawStream(device.index)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        self.held = contextlib.ExitStack()
        if not here:
            self.held.enter_context(torch.cuda.device(device))
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(device.index)
        self.held.enter_context(torch.cuda.stream(stream))
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self.held is not None:
            self.held.close()


def _refuse(t: torch.Tensor, dtype, shape, device, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: must be on {device}, got {t.device}")
    raise ValueError(f"{name}: must be contiguous")


def _need_on(t: torch.Tensor, dtype, shape, device, name) -> int:
    """Data pointer of a contiguous tensor of this type and shape on this device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(t, dtype, shape, device, name)
    return t.data_ptr()


def _need_ws(ws: torch.Tensor, device) -> torch.Tensor:
    if ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: must be a contiguous uint8 tensor on {device}")
    return ws


def _cuda_device(device) -> torch.device:
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("device: must be a CUDA device")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


class _Held:
    """Its tensors' addresses are in a C struct: they are written into, never
    replaced."""

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be replaced; write into the tensor")
        object.__setattr__(self, name, value)


class AdapterPool(_Held):
    """The adapters of one linear as rows of two matrices (the lora_pool_t):
    A (rows x k) and Bt (rows x d, B transposed), bf16.  Adapter a of rank r
    has rows first[a] .. first[a] + r; the rows up to the next multiple of 16
    stay zero.  ``load`` writes an adapter's factors, ``rows_of`` gives its
    slice, for the factors and for the gradients of lora_requests_bwd."""

    def __init__(self, k: int, d: int, ranks, alphas, device=None):
        ranks = [int(r) for r in ranks]
        alphas = [float(a) for a in alphas]
        if not ranks or len(alphas) != len(ranks):
            raise ValueError("one rank and one alpha per adapter, at least one adapter")
        if min(ranks) < 1 or max(ranks) > 256:
            raise ValueError("ranks must lie in 1..256")
        if not all(0.0 < a < float("inf") for a in alphas):
            raise ValueError("alphas must be positive and finite")
        if k < 8 or d < 8 or k % 8 or d % 8:
            raise ValueError("k and d must be positive multiples of 8")
        device = _cuda_device(device)
        self.k, self.d, self.n, self.device = int(k), int(d), len(ranks), device
        self.ranks, self.firsts = ranks, []
        rows = 0
        for r in ranks:
            self.firsts.append(rows)
            rows += (r + 15) // 16 * 16
        self.rows, self.width = rows, (max(ranks) + 15) // 16 * 16
        self.A = torch.zeros(rows, k, dtype=torch.bfloat16, device=device)
        self.Bt = torch.zeros(rows, d, dtype=torch.bfloat16, device=device)
        self.first = torch.tensor(self.firsts, dtype=torch.int32, device=device)
        self.rank = torch.tensor(ranks, dtype=torch.int32, device=device)
        self.scale = torch.tensor([a / r for a, r in zip(alphas, ranks)], dtype=torch.float32, device=device)
        self._c = _Pool(self.A.data_ptr(), self.Bt.data_ptr(), self.first.data_ptr(), self.rank.data_ptr(),
                        self.scale.data_ptr(), rows, k, d, self.n, self.width)
        self._ref = ctypes.byref(self._c)

    @property
    def cstruct(self) -> _Pool:
        return self._c

    def rows_of(self, a: int) -> slice:
        if not 0 <= a < self.n:
            raise IndexError(f"adapter {a} of {self.n}")
        return slice(self.firsts[a], self.firsts[a] + self.ranks[a])

    def load(self, a: int, A: torch.Tensor, B: torch.Tensor) -> None:
        """Adapter a's factors as the layer holds them: A (r x k), B (d x r)."""
        rows, r = self.rows_of(a), self.ranks[a]
        for t, shape, name in ((A, (r, self.k), "A"), (B, (self.d, r), "B")):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != shape:
                raise ValueError(f"{name}: expected bf16 {shape}, got {t.dtype} {tuple(t.shape)}")
        self.A[rows].copy_(A)
        self.Bt[rows].copy_(B.t())


class RequestPlan(_Held):
    """Device buffers of a batch's maps (the lora_requests_t): n_req requests
    over T rows and pools of n adapters; see lora_requests_plan."""

    def __init__(self, n_req: int, n: int, T: int, device=None):
        if n_req < 0 or n < 1 or T < 0:
            raise ValueError("n_req >= 0, n >= 1 and T >= 0")
        tiles = lib().lora_requests_max_tiles(n_req, n, T)
        if tiles <= 0:
            raise ValueError("at most 4096 requests, 4096 adapters and 2^22 rows")
        device = _cuda_device(device)
        self.n_req, self.n, self.T, self.device = int(n_req), int(n), int(T), device

        def ints(count):
            return torch.zeros(max(count, 4), dtype=torch.int32, device=device)[:count]

        self.starts, self.idx, self.order = ints(n_req + 1), ints(T), ints(T)
        self.seg, self._tile_first, self._tiles = ints(n + 2), ints(n + 2), ints(4 * tiles)
        self._c = _Requests(*(t.data_ptr() or self._tiles.data_ptr()
                              for t in (self.starts, self.idx, self.order, self.seg, self._tile_first, self._tiles)),
                            T, n_req, n)
        self._ref = ctypes.byref(self._c)

    @property
    def cstruct(self) -> _Requests:
        return self._c


def lora_requests_plan(lens: torch.Tensor, adapters: torch.Tensor, plan: RequestPlan, stream=None) -> RequestPlan:
    """Fill the plan's maps from the requests' lengths and adapters (int32, device)."""
    lp = _need_on(lens, torch.int32, (plan.n_req,), plan.device, "lens")
    ap = _need_on(adapters, torch.int32, (plan.n_req,), plan.device, "adapters")
    with _On(plan.device, stream) as st:
        _check(lib().lora_requests_plan(lp or plan._tiles.data_ptr(), ap or plan._tiles.data_ptr(),
                                        plan._ref, st), "lora_requests_plan")
    return plan


def _need_match(pool: AdapterPool, plan: RequestPlan):
    if plan.n != pool.n:
        raise ValueError(f"plan for {plan.n} adapters, pool of {pool.n}")
    if plan.device != pool.device:
        raise ValueError(f"plan on {plan.device}, pool on {pool.device}")


def lora_requests_fwd_workspace_bytes(pool: AdapterPool, plan: RequestPlan) -> int:
    return lib().lora_requests_fwd_workspace_bytes(pool._ref, plan._ref)


def lora_requests_bwd_workspace_bytes(pool: AdapterPool, plan: RequestPlan) -> int:
    return lib().lora_requests_bwd_workspace_bytes(pool._ref, plan._ref)


def lora_requests_fwd(pool: AdapterPool, plan: RequestPlan, X: torch.Tensor, base: Optional[torch.Tensor] = None,
                      Y: Optional[torch.Tensor] = None, U_save: Optional[torch.Tensor] = None,
                      save: bool = False, ws: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Y = base + each token's adapter term; with ``save`` (or U_save given)
    also U (T x pool.width, fp32) for the backward.  Y may be ``base``."""
    _need_match(pool, plan)
    dev, T, bf = pool.device, plan.T, torch.bfloat16
    xp = _need_on(X, bf, (T, pool.k), dev, "X")
    bp = None if base is None else _need_on(base, bf, (T, pool.d), dev, "base")
    with _On(dev, stream) as st:
        # rows behind the last request are not written: new outputs start at zero
        Y = torch.zeros(T, pool.d, dtype=bf, device=dev) if Y is None else Y
        if U_save is None and save:
            U_save = torch.zeros(T, pool.width, dtype=torch.float32, device=dev)
        yp = _need_on(Y, bf, (T, pool.d), dev, "Y")
        up = None if U_save is None else _need_on(U_save, torch.float32, (T, pool.width), dev, "U_save")
        ws = workspace(lora_requests_fwd_workspace_bytes(pool, plan), dev) if ws is None else _need_ws(ws, dev)
        _check(lib().lora_requests_fwd(pool._ref, plan._ref, xp, bp, yp, up,
                                       ws.data_ptr(), ws.numel(), st), "lora_requests_fwd")
    return Y, U_save


def lora_requests_bwd(pool: AdapterPool, plan: RequestPlan, X: torch.Tensor, U_saved: torch.Tensor, dY: torch.Tensor,
                      base: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                      dA: Optional[torch.Tensor] = None, dBt: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    """dX = base + the adapters' part, and the gradients of the pool's rows dA
    (rows x k) and dBt (rows x d), fp32."""
    _need_match(pool, plan)
    dev, T, bf, f32 = pool.device, plan.T, torch.bfloat16, torch.float32
    xp = _need_on(X, bf, (T, pool.k), dev, "X")
    up = _need_on(U_saved, f32, (T, pool.width), dev, "U_saved")
    gp = _need_on(dY, bf, (T, pool.d), dev, "dY")
    bp = None if base is None else _need_on(base, bf, (T, pool.k), dev, "base")
    with _On(dev, stream) as st:
        dX = torch.zeros(T, pool.k, dtype=bf, device=dev) if dX is None else dX
        # rows that no entry of the pool's tables names are not written: new gradients start at zero
        dA = torch.zeros(pool.rows, pool.k, dtype=f32, device=dev) if dA is None else dA
        dBt = torch.zeros(pool.rows, pool.d, dtype=f32, device=dev) if dBt is None else dBt
        dxp = _need_on(dX, bf, (T, pool.k), dev, "dX")
        dap = _need_on(dA, f32, (pool.rows, pool.k), dev, "dA")
        dbp = _need_on(dBt, f32, (pool.rows, pool.d), dev, "dBt")
        ws = workspace(lora_requests_bwd_workspace_bytes(pool, plan), dev) if ws is None else _need_ws(ws, dev)
        _check(lib().lora_requests_bwd(pool._ref, plan._ref, xp, up, gp, bp, dxp, dap,
                                       dbp, ws.data_ptr(), ws.numel(), st), "lora_requests_bwd")
    return dX, dA, dBt


def _need_base(q: NF4Weight, pool: AdapterPool):
    if (q.d, q.k) != (pool.d, pool.k):
        raise ValueError(f"weight {q.d} x {q.k}, pool for {pool.d} x {pool.k}")
    if q.codes.device != pool.device:
        raise ValueError(f"weight on {q.codes.device}, pool on {pool.device}")


def qlora_fwd_requests_workspace_bytes(q: NF4Weight, pool: AdapterPool, plan: RequestPlan) -> int:
    return lib().qlora_fwd_requests_workspace_bytes(ctypes.byref(q.cstruct), pool._ref, plan._ref)


def qlora_bwd_requests_workspace_bytes(q: NF4Weight, pool: AdapterPool, plan: RequestPlan) -> int:
    return lib().qlora_bwd_requests_workspace_bytes(ctypes.byref(q.cstruct), pool._ref, plan._ref)


def qlora_fwd_requests(q: NF4Weight, pool: AdapterPool, plan: RequestPlan, X: torch.Tensor,
                       Y: Optional[torch.Tensor] = None, U_save: Optional[torch.Tensor] = None, save: bool = False,
                       ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The layer on the NF4 weight with each request's adapter: Y, and U for
    the backward with ``save`` (or U_save given)."""
    _need_match(pool, plan)
    _need_base(q, pool)
    dev, T, bf = pool.device, plan.T, torch.bfloat16
    xp = _need_on(X, bf, (T, pool.k), dev, "X")
    with _On(dev, stream) as st:
        Y = torch.empty(T, pool.d, dtype=bf, device=dev) if Y is None else Y
        if U_save is None and save:
            U_save = torch.zeros(T, pool.width, dtype=torch.float32, device=dev)
        yp = _need_on(Y, bf, (T, pool.d), dev, "Y")
        up = None if U_save is None else _need_on(U_save, torch.float32, (T, pool.width), dev, "U_save")
        ws = workspace(qlora_fwd_requests_workspace_bytes(q, pool, plan), dev) if ws is None else _need_ws(ws, dev)
        _check(lib().qlora_fwd_requests(ctypes.byref(q.cstruct), pool._ref, plan._ref, xp, yp, up, ws.data_ptr(),
                                        ws.numel(), st), "qlora_fwd_requests")
    return Y, U_save


def qlora_bwd_requests(q: NF4Weight, pool: AdapterPool, plan: RequestPlan, X: torch.Tensor, U_saved: torch.Tensor,
                       dY: torch.Tensor, dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                       dBt: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of qlora_fwd_requests: dX, and dA (rows x k), dBt (rows x d) of the pool's rows."""
    _need_match(pool, plan)
    _need_base(q, pool)
    dev, T, bf, f32 = pool.device, plan.T, torch.bfloat16, torch.float32
    xp = _need_on(X, bf, (T, pool.k), dev, "X")
    up = _need_on(U_saved, f32, (T, pool.width), dev, "U_saved")
    gp = _need_on(dY, bf, (T, pool.d), dev, "dY")
    with _On(dev, stream) as st:
        dX = torch.empty(T, pool.k, dtype=bf, device=dev) if dX is None else dX
        # rows that no entry of the pool's tables names are not written: new gradients start at zero
        dA = torch.zeros(pool.rows, pool.k, dtype=f32, device=dev) if dA is None else dA
        dBt = torch.zeros(pool.rows, pool.d, dtype=f32, device=dev) if dBt is None else dBt
        dxp = _need_on(dX, bf, (T, pool.k), dev, "dX")
        dap = _need_on(dA, f32, (pool.rows, pool.k), dev, "dA")
        dbp = _need_on(dBt, f32, (pool.rows, pool.d), dev, "dBt")
        ws = workspace(qlora_bwd_requests_workspace_bytes(q, pool, plan), dev) if ws is None else _need_ws(ws, dev)
        _check(lib().qlora_bwd_requests(ctypes.byref(q.cstruct), pool._ref, plan._ref, xp, up, gp, dxp, dap, dbp,
                                        ws.data_ptr(), ws.numel(), st), "qlora_bwd_requests")
    return dX, dA, dBt


def lora_muon_workspace_bytes(n: int, rows: int, cols: int) -> int:
    return lib().lora_muon_workspace_bytes(n, rows, cols)


def lora_muon_step(master: torch.Tensor, weight_bf16: torch.Tensor, m: torch.Tensor, grad: torch.Tensor, lr: float,
                   momentum: float = 0.95, nesterov: bool = True, scale: float = 1.0, weight_decay: float = 0.0,
                   eps: float = 1e-7, steps: int = 5, coefs=None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """One step that orthogonalises the momentum of each matrix of a stack
    (n x rows x cols, or one rows x cols), in place on (master, m) and the
    bf16 copy; see qlora.h.  At most 8 steps with the usual coefs (in general
    |coefs[0]| ** (2 * steps) <= 2 ** 30)."""
    if master.dim() not in (2, 3):
        raise ValueError("master: expected rows x cols or n x rows x cols")
    n = 1 if master.dim() == 2 else master.shape[0]
    rows, cols = master.shape[-2], master.shape[-1]
    dev = master.device
    if n == 0:
        return
    if dev.type != "cuda":
        raise ValueError("master: must be a CUDA tensor")
    ptrs = [_need_on(t, dt, master.shape, dev, name)
            for t, dt, name in ((master, torch.float32, "master"), (weight_bf16, torch.bfloat16, "weight_bf16"),
                                (m, torch.float32, "m"), (grad, torch.float32, "grad"))]
    cs = None
    if coefs is not None:
        if len(coefs) != 3:
            raise ValueError("coefs: expected three")
        cs = (ctypes.c_float * 3)(*[float(c) for c in coefs])
    with _On(dev, stream) as st:
        ws = workspace(lora_muon_workspace_bytes(n, rows, cols), dev) if ws is None else _need_ws(ws, dev)
        _check(lib().lora_muon_step(*ptrs, n, rows, cols, float(lr), float(momentum), int(bool(nesterov)), float(scale),
                                    float(weight_decay), float(eps), int(steps),
                                    None if cs is None else ctypes.addressof(cs), ws.data_ptr(), ws.numel(), st),
               "lora_muon_step")


def lora_merge(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
               W_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    r = A.shape[0]
    _need(A, torch.bfloat16, (r, q.k), "A")
    _need(B, torch.bfloat16, (q.d, r), "B")
    W_out = torch.empty(q.d, q.k, dtype=torch.bfloat16, device=A.device) if W_out is None else W_out
    _need(W_out, torch.bfloat16, (q.d, q.k), "W_out")
    nbytes = lora_merge_workspace_bytes(q.d, q.k, r)
    ws = workspace(nbytes, A.device) if ws is None else ws
    st = lib().lora_merge(ctypes.byref(q.cstruct), _ptr(A), _ptr(B), r, float(alpha), _ptr(W_out),
                          _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lora_merge")
    return W_out


def lora_unmerge(W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                 W0_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    d, k = W.shape
    r = A.shape[0]
    _need(W, torch.bfloat16, (d, k), "W")
    _need(A, torch.bfloat16, (r, k), "A")
    _need(B, torch.bfloat16, (d, r), "B")
    W0_out = torch.empty(d, k, dtype=torch.bfloat16, device=W.device) if W0_out is None else W0_out
    _need(W0_out, torch.bfloat16, (d, k), "W0_out")
    nbytes = lora_merge_workspace_bytes(d, k, r)
    ws = workspace(nbytes, W.device) if ws is None else ws
    st = lib().lora_unmerge(_ptr(W), _ptr(A), _ptr(B), r, float(alpha), d, k, _ptr(W0_out),
                            _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lora_unmerge")
    return W0_out


def qlora_get_device_status(stream=None) -> int:
    v = ctypes.c_int(0)
    _check(lib().qlora_get_device_status(_stream(stream), ctypes.byref(v)), "qlora_get_device_status")
    return v.value


def qlora_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib().qlora_selftest_wait_timeout(int(limit_us), _stream(stream)), "qlora_selftest_wait_timeout")


# ------------------------------------------------------------------ data parallel
NCCL_ID_BYTES = 128


def qlora_comm_unique_id() -> bytes:
    """A new NCCL unique id for the caller to share with every rank."""
    buf = (ctypes.c_uint8 * NCCL_ID_BYTES)()
    _check(lib().qlora_comm_unique_id(ctypes.addressof(buf)), "qlora_comm_unique_id")
    return bytes(buf)


class Communicator:
    """This rank's NCCL communicator for the adapter-gradient sum (owned by
    the caller; release it with close() after its last collective)."""

    def __init__(self, unique_id: bytes, nranks: int, rank: int):
        if len(unique_id) != NCCL_ID_BYTES:
            raise ValueError(f"unique_id must be {NCCL_ID_BYTES} bytes")
        buf = (ctypes.c_uint8 * NCCL_ID_BYTES).from_buffer_copy(unique_id)
        h = ctypes.c_void_p()
        _check(lib().qlora_comm_init(ctypes.addressof(buf), int(nranks), int(rank), ctypes.byref(h)),
               "qlora_comm_init")
        self.handle = h.value
        self.nranks, self.rank = nranks, rank

    def close(self) -> None:
        if self.handle:
            _check(lib().qlora_comm_destroy(self.handle), "qlora_comm_destroy")
            self.handle = None


def communicator_from_process_group(group=None, make=Communicator):
    """This rank's communicator over the ranks of a torch.distributed group:
    rank 0 draws the NCCL id and the group broadcasts it (any backend)."""
    import torch.distributed as dist
    rank, n = dist.get_rank(group), dist.get_world_size(group)
    box = [qlora_comm_unique_id() if rank == 0 else None]
    dist.broadcast_object_list(box, src=dist.get_global_rank(group, 0) if group is not None else 0, group=group)
    return make(box[0], n, rank)


def qlora_grad_allreduce(comm: "Communicator", dA: torch.Tensor, dB: torch.Tensor, stream=None) -> None:
    """dA and dB (fp32, device) become their sums over the ranks, in place."""
    for name, t in (("dA", dA), ("dB", dB)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    _check(lib().qlora_grad_allreduce(comm.handle, _ptr(dA), dA.numel(), _ptr(dB), dB.numel(), _stream(stream)),
           "qlora_grad_allreduce")


def qlora_profile_begin() -> None:
    _check(lib().qlora_profile_begin(), "qlora_profile_begin")


def qlora_profile_end():
    cap = 64
    arr = (KernelStat * cap)()
    n = ctypes.c_int(0)
    _check(lib().qlora_profile_end(arr, cap, ctypes.byref(n)), "qlora_profile_end")
    return [{"name": arr[i].name.decode(), "launches": arr[i].launches, "total_ms": arr[i].total_ms,
             "flops": arr[i].flops, "bytes": arr[i].bytes} for i in range(min(n.value, cap))]
