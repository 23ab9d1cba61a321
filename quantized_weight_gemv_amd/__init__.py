"""Python binding of libqgemv.so (gfx950): fused dequantize-and-multiply of
block-quantized weights (Q4_0, Q8_0, plain 2-bit q2w and 8-bit floating f8),
8-bit activation checkpoints with the products of the backward pass, and
expert routing.

This module only marshals arguments: it checks tensor devices, dtypes, shapes
and sizes (the C ABI cannot see buffer sizes), passes raw pointers and the
current HIP stream, and turns a non-zero status into an exception.  Every step
of the computation runs in the library's HIP kernels; there is no fallback.
Autograd records none of the calls.  The f8 and routing calls, which have
gradients of their own to be put together, refuse tensors that require one while
gradients are recorded; torch.autograd.Function's forward and backward run
without.
If the library is missing the import of any entry point fails loudly.

Names follow the C ABI in include/qgemv.h and include/qgemv_f8.h.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# QGEMV_LIB points the binding at another build of the library (for example
# a variant compiled for an experiment); default: the in-tree build.
LIB_PATH = os.environ.get("QGEMV_LIB") or os.path.join(_HERE, "libqgemv.so")

QG_STATUS = {0: "ok", 1: "null pointer", 2: "shape out of range", 3: "misaligned pointer",
             4: "non-finite weight or scale overflow", 5: "buffer too small", 6: "kernel launch failed",
             7: "no usable HIP device"}

Q4_0 = 0
Q8_0 = 1
Q2W = 2


class QGError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: status {status} ({QG_STATUS.get(status, 'unknown')})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqgemv.so (after torch, so both use the one HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -m quantized_weight_gemv_amd.build` "
                          f"(or __graft_entry__.build())")
    try:
        import torch  # noqa: F401  (loads the HIP runtime the library must share)
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    sig = {
        "qg_status_str": (ctypes.c_char_p, [c_int]),
        "qpacked_bytes_q4_0": (sz, [i64, i64]),
        "qpacked_bytes_q8_0": (sz, [i64, i64]),
        "qquantize_q4_0": (c_int, [vp, i64, i64, vp, sz]),
        "qquantize_q8_0": (c_int, [vp, i64, i64, vp, sz]),
        "qpacked_bytes_q2w": (sz, [i64, i64]),
        "qquantize_q2w": (c_int, [vp, i64, i64, vp, sz]),
        "qgemv_q2w": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q2w_q8act": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q2w_lut": (c_int, [vp, vp, vp, i64, i64, vp]),
        "qdequant_q2w": (c_int, [vp, i64, i64, c_int, vp, vp]),
        "qgemv_q4_0": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q8_0": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q4_0_f32in": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q4_0_swiglu_f32in": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qgemv_q4_0_q8act": (c_int, [vp, vp, vp, c_int, i64, i64, vp]),
        "qmoe_gemv_q4_0": (c_int, [vp, i64, vp, vp, vp, c_int, i64, i64, vp]),
        "qgemm_q4_0_prefill": (c_int, [vp, vp, vp, i64, i64, i64, vp]),
        "qdequant_q4_0": (c_int, [vp, i64, i64, c_int, vp, vp]),
        "qdequant_q8_0": (c_int, [vp, i64, i64, c_int, vp, vp]),
        "qpacked_bytes_f8": (sz, [i64, i64]),
        "qact_bytes_f8": (sz, [i64, i64]),
        "qquantize_f8": (c_int, [vp, i64, i64, vp, sz]),
        "qdequant_f8": (c_int, [vp, i64, i64, c_int, vp, vp]),
        "qtranspose_f8": (c_int, [vp, i64, i64, vp, vp]),
        "qact_quantize_f8": (c_int, [vp, c_int, i64, i64, i64, vp, vp]),
        "qact_dequant_f8": (c_int, [vp, i64, i64, c_int, vp, vp]),
        "qgemv_f8": (c_int, [vp, vp, c_int, vp, c_int, i64, i64, vp]),
        "qgemm_f8": (c_int, [vp, vp, vp, c_int, i64, i64, i64, vp]),
        "qgemm_f8_wgrad_workspace": (sz, [i64, i64, i64]),
        "qgemm_f8_wgrad": (c_int, [vp, vp, vp, c_int, i64, i64, i64, vp, vp]),
        "qmoe_route_workspace": (sz, [i64, i64]),
        "qmoe_route": (c_int, [vp, c_int, i64, vp, i64, i64, c_int, c_int, vp, vp, vp, vp, vp, vp, vp, vp]),
        "qmoe_route_backward": (c_int, [vp, c_int, i64, vp, i64, i64, c_int, c_int, vp, vp, vp, vp, vp, vp, vp]),
        "qmoe_gemm_f8": (c_int, [vp, i64, vp, i64, c_int, vp, vp, vp, c_int, i64, i64, vp]),
        "qmoe_gemm_f8_wgrad": (c_int, [vp, vp, i64, c_int, vp, vp, i64, vp, c_int, i64, i64, vp]),
        "qg_time_next_launch": (None, [vp, vp]),
        "qg_device_cus": (c_int, [c_int, ctypes.POINTER(c_int)]),
        "qg_set_gemv_shape": (None, [c_int, c_int, c_int, c_int, i64, c_int, c_int, c_int]),
        "qg_read_probe": (c_int, [vp, sz, vp, c_int, c_int, vp]),
        "qg_set_prefill_shape": (None, [c_int, c_int]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def exported_symbols() -> list[str]:
    return ["qg_status_str", "qpacked_bytes_q4_0", "qpacked_bytes_q8_0", "qquantize_q4_0", "qquantize_q8_0",
            "qgemv_q4_0", "qgemv_q8_0", "qgemv_q4_0_f32in", "qgemv_q4_0_swiglu_f32in", "qgemv_q4_0_q8act",
            "qmoe_gemv_q4_0",
            "qgemm_q4_0_prefill", "qdequant_q4_0",
            "qdequant_q8_0", "qpacked_bytes_q2w", "qquantize_q2w", "qgemv_q2w", "qgemv_q2w_q8act", "qgemv_q2w_lut", "qdequant_q2w",
            "qpacked_bytes_f8", "qact_bytes_f8", "qquantize_f8", "qdequant_f8", "qtranspose_f8", "qact_quantize_f8",
            "qact_dequant_f8", "qgemv_f8", "qgemm_f8", "qgemm_f8_wgrad_workspace", "qgemm_f8_wgrad",
            "qmoe_route_workspace", "qmoe_route", "qmoe_route_backward", "qmoe_gemm_f8", "qmoe_gemm_f8_wgrad",
            "qg_time_next_launch", "qg_device_cus", "qg_set_gemv_shape", "qg_read_probe", "qg_set_prefill_shape"]


def _check(fn: str, st: int):
    if st != 0:
        raise QGError(fn, st)


# ------------------------------------------------------------------ host side
def qpacked_bytes_q4_0(N: int, K: int) -> int:
    return int(lib().qpacked_bytes_q4_0(N, K))


def qpacked_bytes_q8_0(N: int, K: int) -> int:
    return int(lib().qpacked_bytes_q8_0(N, K))


def qpacked_bytes_q2w(N: int, K: int) -> int:
    return int(lib().qpacked_bytes_q2w(N, K))


def packed_bytes(fmt: int, N: int, K: int) -> int:
    if fmt == Q2W:
        return qpacked_bytes_q2w(N, K)
    return qpacked_bytes_q4_0(N, K) if fmt == Q4_0 else qpacked_bytes_q8_0(N, K)


def _quantize(fn: str, fmt: int, w: np.ndarray, out: np.ndarray | None) -> np.ndarray:
    w = np.ascontiguousarray(w, dtype=np.float32)
    if w.ndim != 2:
        raise ValueError("weights must be [N][K]")
    N, K = w.shape
    nb = packed_bytes(fmt, N, K)
    if nb == 0:
        raise QGError(fn, 2)
    if out is None:
        out = np.empty(nb, np.uint8)
    if out.dtype != np.uint8 or not out.flags["C_CONTIGUOUS"] or out.size < nb:
        raise ValueError("out must be a contiguous uint8 array of at least the packed size")
    _check(fn, getattr(lib(), fn)(w.ctypes.data, N, K, out.ctypes.data, out.size))
    return out


def qquantize_q4_0(w: np.ndarray, out: np.ndarray | None = None) -> np.ndarray:
    """Quantize + pack fp32 [N][K] host weights into the Q4_0 layout (host bytes)."""
    return _quantize("qquantize_q4_0", Q4_0, w, out)


def qquantize_q8_0(w: np.ndarray, out: np.ndarray | None = None) -> np.ndarray:
    """Quantize + pack fp32 [N][K] host weights into the Q8_0 layout (host bytes)."""
    return _quantize("qquantize_q8_0", Q8_0, w, out)


def qquantize_q2w(w: np.ndarray, out: np.ndarray | None = None) -> np.ndarray:
    """Quantize + pack fp32 [N][K] host weights into the plain 2-bit (q2w) layout."""
    return _quantize("qquantize_q2w", Q2W, w, out)


# ---------------------------------------------------------------- device side
def _torch():
    import torch
    return torch


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _dev(t, dtype, name: str, numel: int | None = None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _x16(x):
    torch = _torch()
    if x.dtype == torch.float16:
        return x.view(torch.int16)
    return x


def _gemv(fn: str, fmt: int, Wp, x, N: int, K: int, y=None):
    torch = _torch()
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M][{K}]")
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    wp = _dev(Wp, torch.uint8, "Wp", packed_bytes(fmt, N, K))
    xp = _dev(_x16(x), torch.int16, "x", M * K)
    yp = _dev(y, torch.float32, "y", M * N)
    _check(fn, getattr(lib(), fn)(wp, xp, yp, M, N, K, _stream()))
    return y


class PreparedGemv:
    """A qgemv_* call validated once, for launch-bound loops: calling it only
    enqueues the kernel (ctypes call with the stored raw pointers) on the
    stream that was current when it was prepared.  The tensors must stay
    alive and unmoved while the object is used."""

    def __init__(self, fmt: int, Wp, x, y, N: int, K: int):
        torch = _torch()
        if x.dim() != 2 or x.shape[1] != K or y.shape != (x.shape[0], N):
            raise ValueError("x must be [M][K] and y [M][N]")
        self._keep = (Wp, x, y)
        self._name = {Q4_0: "qgemv_q4_0", Q8_0: "qgemv_q8_0", Q2W: "qgemv_q2w"}[fmt]
        self._fn = getattr(lib(), self._name)
        self._args = (_dev(Wp, torch.uint8, "Wp", packed_bytes(fmt, N, K)).value,
                      _dev(_x16(x), torch.int16, "x", x.shape[0] * K).value,
                      _dev(y, torch.float32, "y", x.shape[0] * N).value,
                      int(x.shape[0]), int(N), int(K), _stream().value)

    def __call__(self):
        st = self._fn(*self._args)
        if st:
            raise QGError(self._name, st)


def qgemv_q4_0(Wp, x, N: int, K: int, y=None):
    """y[M][N] (fp32) = dequant(Wp) @ x[M][K]^T; Wp uint8 packed Q4_0, x fp16, 1 <= M <= 8."""
    return _gemv("qgemv_q4_0", Q4_0, Wp, x, N, K, y)


def qgemv_q8_0(Wp, x, N: int, K: int, y=None):
    """y[M][N] (fp32) = dequant(Wp) @ x[M][K]^T; Wp uint8 packed Q8_0, x fp16, 1 <= M <= 8."""
    return _gemv("qgemv_q8_0", Q8_0, Wp, x, N, K, y)


def qgemv_q2w(Wp, x, N: int, K: int, y=None):
    """y[M][N] (fp32) = dequant(Wp) @ x[M][K]^T; Wp uint8 packed q2w, x fp16, 1 <= M <= 8."""
    return _gemv("qgemv_q2w", Q2W, Wp, x, N, K, y)


def qgemv_q2w_q8act(Wp, x, N: int, K: int, y=None):
    """y[M][N] = q2w weights times fp16 x quantized to 8-bit blocks inside the
    launch (int8 dot products); 1 <= M <= 4."""
    return _gemv("qgemv_q2w_q8act", Q2W, Wp, x, N, K, y)


def qgemv_q2w_lut(Wp, x, N: int, K: int, y=None):
    """y[1][N] = q2w weights times one fp16 token through per-pair lookup
    tables in LDS (the times-table design); K <= 4096."""
    torch = _torch()
    if x.dim() != 2 or x.shape != (1, K):
        raise ValueError(f"x must be [1][{K}]")
    if y is None:
        y = torch.empty((1, N), dtype=torch.float32, device=x.device)
    wp = _dev(Wp, torch.uint8, "Wp", packed_bytes(Q2W, N, K))
    xp = _dev(_x16(x), torch.int16, "x", K)
    yp = _dev(y, torch.float32, "y", N)
    _check("qgemv_q2w_lut", lib().qgemv_q2w_lut(wp, xp, yp, N, K, _stream()))
    return y


def qgemv_q4_0_q8act(Wp, x, N: int, K: int, y=None):
    """y[M][N] = Q4_0 weights times fp16 x quantized to 8-bit blocks inside the
    launch (int8 dot products); 1 <= M <= 4."""
    return _gemv("qgemv_q4_0_q8act", Q4_0, Wp, x, N, K, y)


def _f32in(fn: str, Wp, x, N: int, K: int, y, rows: int):
    torch = _torch()
    if x.dim() != 2 or x.shape[1] != K or x.dtype != torch.float32:
        raise ValueError(f"x must be float32 [M][{K}]")
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    wp = _dev(Wp, torch.uint8, "Wp", qpacked_bytes_q4_0(rows, K))
    xp = _dev(x, torch.float32, "x", M * K)
    yp = _dev(y, torch.float32, "y", M * N)
    _check(fn, getattr(lib(), fn)(wp, xp, yp, M, N, K, _stream()))
    return y


def qgemv_q4_0_f32in(Wp, x, N: int, K: int, y=None):
    """y[M][N] = dequant(Wp) @ fp16(x)^T with fp32 x rounded inside the kernel; 1 <= M <= 8."""
    return _f32in("qgemv_q4_0_f32in", Wp, x, N, K, y, N)


def qgemv_q4_0_swiglu_f32in(Wp, x, N: int, K: int, y=None):
    """y[M][N] = silu(gate) * up; Wp packs the 2N x K table [gate rows; up rows]."""
    return _f32in("qgemv_q4_0_swiglu_f32in", Wp, x, N, K, y, 2 * N)


def qmoe_gemv_q4_0(pool, P: int, idx, x, N: int, K: int, y=None):
    """y[E][N] = expert idx[e] of the pool times token x[e]; one launch."""
    torch = _torch()
    E = idx.numel()
    if x.dim() != 2 or x.shape != (E, K):
        raise ValueError(f"x must be [E={E}][{K}]")
    if y is None:
        y = torch.empty((E, N), dtype=torch.float32, device=x.device)
    pp = _dev(pool, torch.uint8, "pool", P * qpacked_bytes_q4_0(N, K))
    ip = _dev(idx, torch.int32, "idx", E)
    xp = _dev(_x16(x), torch.int16, "x", E * K)
    yp = _dev(y, torch.float32, "y", E * N)
    _check("qmoe_gemv_q4_0", lib().qmoe_gemv_q4_0(pp, P, ip, xp, yp, E, N, K, _stream()))
    return y


def qgemm_q4_0_prefill(Wp, X, N: int, K: int, Y=None):
    """Y[M][N] (fp32) = X[M][K] @ dequant(Wp)^T on fp16 matrix cores."""
    torch = _torch()
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"X must be [M][{K}]")
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    wp = _dev(Wp, torch.uint8, "Wp", qpacked_bytes_q4_0(N, K))
    xp = _dev(_x16(X), torch.int16, "X", M * K)
    yp = _dev(Y, torch.float32, "Y", M * N)
    _check("qgemm_q4_0_prefill", lib().qgemm_q4_0_prefill(wp, xp, yp, M, N, K, _stream()))
    return Y


def _dequant(fn: str, fmt: int, Wp, N: int, K: int, fp16: bool, out=None):
    torch = _torch()
    dt = torch.float16 if fp16 else torch.float32
    if out is None:
        out = torch.empty((N, K), dtype=dt, device=Wp.device)
    wp = _dev(Wp, torch.uint8, "Wp", packed_bytes(fmt, N, K))
    op = _dev(out, dt, "out", N * K)
    _check(fn, getattr(lib(), fn)(wp, N, K, 1 if fp16 else 0, op, _stream()))
    return out


def qdequant_q4_0(Wp, N: int, K: int, fp16: bool = False, out=None):
    return _dequant("qdequant_q4_0", Q4_0, Wp, N, K, fp16, out)


def qdequant_q8_0(Wp, N: int, K: int, fp16: bool = False, out=None):
    return _dequant("qdequant_q8_0", Q8_0, Wp, N, K, fp16, out)


def qdequant_q2w(Wp, N: int, K: int, fp16: bool = False, out=None):
    return _dequant("qdequant_q2w", Q2W, Wp, N, K, fp16, out)


# ------------------------------------------------------------------------- f8
def qpacked_bytes_f8(N: int, K: int) -> int:
    """Bytes of one packed N x K f8 matrix (0 where the sizes are out of range)."""
    return int(lib().qpacked_bytes_f8(N, K))


def qact_bytes_f8(M: int, K: int) -> int:
    """Bytes of M x K packed f8 activations (0 where the sizes are out of range)."""
    return int(lib().qact_bytes_f8(M, K))


def qquantize_f8(w: np.ndarray, out: np.ndarray | None = None) -> np.ndarray:
    """Quantize + pack fp32 [N][K] host weights into the f8 layout (host bytes)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    if w.ndim != 2:
        raise ValueError("weights must be [N][K]")
    N, K = w.shape
    nb = qpacked_bytes_f8(N, K)
    if nb == 0:
        raise QGError("qquantize_f8", 2)
    if out is None:
        out = np.empty(nb, np.uint8)
    if out.dtype != np.uint8 or not out.flags["C_CONTIGUOUS"] or out.size < nb:
        raise ValueError("out must be a contiguous uint8 array of at least the packed size")
    _check("qquantize_f8", lib().qquantize_f8(w.ctypes.data, N, K, out.ctypes.data, out.size))
    return out


def _type(dtype) -> int:
    """QG_F32 / QG_F16 / QG_BF16 of a torch dtype."""
    torch = _torch()
    code = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    return code


class _Call:
    """One call's device: every tensor has to be on it, and the call is made
    with it as the current device, on its current stream."""

    __slots__ = ("device", "index", "torch")

    def __init__(self, first, name: str):
        self.torch = torch = _torch()
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError(f"{name} must be a device tensor")
        if first.requires_grad:
            self.no_grad(name)
        self.device = first.device
        self.index = first.get_device()

    def no_grad(self, name: str):
        # the calls are not recorded: an output without a gradient would end the backward pass unseen
        if self.torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, which this call would not pass on: make it under "
                             "torch.no_grad() or inside a torch.autograd.Function")

    def ptr(self, t, dtype, name: str, numel: int):
        # one pass over what has to hold; the reasons are looked up only for a refusal
        if isinstance(t, self.torch.Tensor) and t.get_device() == self.index and t.dtype is dtype and \
                t.numel() >= numel and t.is_contiguous():
            if t.requires_grad:
                self.no_grad(name)
            return t.data_ptr()
        if not isinstance(t, self.torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a device tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")

    def opt(self, t, dtype, name: str, numel: int):
        return None if t is None else self.ptr(t, dtype, name, numel)

    def new(self, shape, dtype):
        return self.torch.empty(shape, dtype=dtype, device=self.device)

    def result(self, t, shape, dtype, name: str, numel: int):
        """The caller's output of this shape, or a new one, and its address."""
        if t is None:
            t = self.torch.empty(shape, dtype=dtype, device=self.device)
            return t, t.data_ptr()
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        return t, self.ptr(t, dtype, name, numel)

    def __call__(self, fn: str, *args):
        f = getattr(lib(), fn)
        index = self.index
        # the stream's handle as it is: torch.cuda.current_stream() makes an
        # object around it first (2.7 us of the 9.7 that a small call took)
        stream = self.torch._C._cuda_getCurrentRawStream(index)
        if index == self.torch.cuda.current_device():
            st = f(*args, stream)
        else:
            with self.torch.cuda.device(index):
                st = f(*args, stream)
        if st:
            raise QGError(fn, st)


def _sizes(fn: str, *nbytes: int):
    if 0 in nbytes:
        raise QGError(fn, 2)


def qdequant_f8(Wp, N: int, K: int, fp16: bool = False, out=None):
    """The values of a packed f8 matrix, [N][K] in fp32 or fp16."""
    c, nb = _Call(Wp, "Wp"), qpacked_bytes_f8(N, K)
    _sizes("qdequant_f8", nb)
    out, op = c.result(out, (N, K), c.torch.float16 if fp16 else c.torch.float32, "out", N * K)
    c("qdequant_f8", c.ptr(Wp, c.torch.uint8, "Wp", nb), N, K, int(fp16), op)
    return out


def qtranspose_f8(Wp, N: int, K: int, out=None):
    """The packed N x K matrix as the packed K x N matrix (exact), the operand of dx = f8(dy) W."""
    c, nb, nt = _Call(Wp, "Wp"), qpacked_bytes_f8(N, K), qpacked_bytes_f8(K, N)
    _sizes("qtranspose_f8", nb, nt)
    if out is None:
        out = c.new((nt,), c.torch.uint8)
    c("qtranspose_f8", c.ptr(Wp, c.torch.uint8, "Wp", nb), N, K, c.ptr(out, c.torch.uint8, "out", nt))
    return out


def qact_quantize_f8(x, out=None):
    """x[M][K] (fp32, fp16 or bf16; rows may be strided) -> packed f8 activations (uint8)."""
    c = _Call(x, "x")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be [M][K] with contiguous rows")
    M, K = x.shape
    nb = qact_bytes_f8(M, K)
    _sizes("qact_quantize_f8", nb)
    if out is None:
        out = c.new((nb,), c.torch.uint8)
        op = out.data_ptr()
    else:
        op = c.ptr(out, c.torch.uint8, "out", nb)
    c("qact_quantize_f8", x.data_ptr(), _type(x.dtype), x.stride(0) if M > 1 else K, M, K, op)
    return out


def qact_dequant_f8(xq, M: int, K: int, dtype=None, out=None):
    """The values of packed f8 activations, [M][K] (fp32 by default)."""
    c, nb = _Call(xq, "xq"), qact_bytes_f8(M, K)
    _sizes("qact_dequant_f8", nb)
    dtype = dtype or (c.torch.float32 if out is None else out.dtype)
    code = _type(dtype)
    out, op = c.result(out, (M, K), dtype, "out", M * K)
    c("qact_dequant_f8", c.ptr(xq, c.torch.uint8, "xq", nb), M, K, code, op)
    return out


def qgemv_f8(Wp, x, N: int, K: int, y=None):
    """y[M][N] (fp32) = f8(x)[M][K] @ W^T, 1 <= M <= 8: x (fp32, fp16 or bf16) is quantized inside the launch."""
    c, nb = _Call(Wp, "Wp"), qpacked_bytes_f8(N, K)
    _sizes("qgemv_f8", nb)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M][{K}]")
    M = x.shape[0]
    y, yp = c.result(y, (M, N), c.torch.float32, "y", M * N)
    c("qgemv_f8", c.ptr(Wp, c.torch.uint8, "Wp", nb), c.ptr(x, x.dtype, "x", M * K), _type(x.dtype), yp, M, N, K)
    return y


def qgemm_f8(Wp, xq, M: int, N: int, K: int, dtype=None, Y=None):
    """Y[M][N] = X @ W^T on packed f8 activations (fp32 by default, or fp16 / bf16)."""
    c, nb, na = _Call(Wp, "Wp"), qpacked_bytes_f8(N, K), qact_bytes_f8(M, K)
    _sizes("qgemm_f8", nb, na)
    dtype = dtype or (c.torch.float32 if Y is None else Y.dtype)
    code = _type(dtype)
    Y, yp = c.result(Y, (M, N), dtype, "Y", M * N)
    u8 = c.torch.uint8
    c("qgemm_f8", c.ptr(Wp, u8, "Wp", nb), c.ptr(xq, u8, "xq", na), yp, code, M, N, K)
    return Y


def qgemm_f8_wgrad(dY, xq, M: int, N: int, K: int, dW=None, accumulate: bool = False):
    """dW[N][K] (fp32) = dY[M][N]^T @ X from bf16 dY and the packed f8 activations X (added to dW with accumulate)."""
    c, na = _Call(dY, "dY"), qact_bytes_f8(M, K)
    _sizes("qgemm_f8_wgrad", na, qpacked_bytes_f8(N, K))
    if accumulate and dW is None:
        raise ValueError("accumulate needs dW")
    dW, wp = c.result(dW, (N, K), c.torch.float32, "dW", N * K)
    ws = int(lib().qgemm_f8_wgrad_workspace(M, N, K))
    w = c.new((ws,), c.torch.uint8) if ws else None
    c("qgemm_f8_wgrad", c.ptr(dY, c.torch.bfloat16, "dY", M * N), c.ptr(xq, c.torch.uint8, "xq", na), wp,
      int(accumulate), M, N, K, w.data_ptr() if ws else None)
    return dW


class MoeRoute(NamedTuple):
    """What qmoe_route returns; qmoe_route_backward and qmoe_gemm_f8 take it up."""
    idx: object       # int32 [T][k], -1: no expert
    weight: object    # fp32 [T][k]
    counts: object    # int32 [E], slots of each expert
    tokens: object    # int32 [1], tokens that were routed
    offsets: object   # int32 [E + 1]
    order: object     # int32 [T k], the slots sorted by expert
    loss: object      # fp32 [1], the balance loss


def _logits(logits, mask):
    torch = _torch()
    c = _Call(logits, "logits")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T][E] with contiguous rows")
    T, E = logits.shape
    if mask is not None and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    if mask is not None and mask.shape != (T,):
        raise ValueError(f"mask must be [{T}]")
    return c, T, E, logits.stride(0) if T > 1 else E, c.opt(mask, torch.uint8, "mask", T)


def qmoe_route(logits, k: int, mask=None, renormalize: bool = True) -> MoeRoute:
    """Top-k softmax routing of logits[T][E] (fp32, fp16 or bf16; rows may be
    strided) with per-expert counts, the slots sorted by expert and the balance
    loss; mask (bool or uint8 [T]): 0 for tokens that are not routed."""
    torch = _torch()
    c, T, E, ld, mp = _logits(logits, mask)
    code = _type(logits.dtype)
    if not (1 <= k <= min(E, 16) and 1 <= T <= 1 << 24 and E <= 512):
        raise QGError("qmoe_route", 2)
    # one buffer a type: tensors are made faster by splitting one (0.4 us each) than one by one (1.5)
    S = T * k
    ints, floats = c.new((2 * S + 2 * E + 2,), torch.int32), c.new((S + 1,), torch.float32)
    ip, fp = ints.data_ptr(), floats.data_ptr()
    ws = int(lib().qmoe_route_workspace(T, E))
    w = c.new((ws,), torch.uint8) if ws else None
    c("qmoe_route", logits.data_ptr(), code, ld, mp, T, E, k, int(renormalize), ip, fp, ip + 8 * S,
      ip + 8 * S + 4 * (E + 1), ip + 4 * S, fp + 4 * S, w.data_ptr() if ws else None)
    idx, order, counts, tokens, offsets = ints.split_with_sizes((S, S, E, 1, E + 1))
    weight, loss = floats.split_with_sizes((S, 1))
    idx, weight = idx.view(T, k), weight.view(T, k)
    return MoeRoute(idx, weight, counts, tokens, offsets, order, loss)


def qmoe_route_backward(logits, route: MoeRoute, grad_weight=None, grad_loss=None, mask=None,
                        renormalize: bool = True, out=None):
    """The gradient of route.weight and route.loss with respect to the logits (their type)."""
    torch = _torch()
    c, T, E, ld, mp = _logits(logits, mask)
    k = route.idx.shape[1]
    if route.idx.shape != (T, k) or route.weight.shape != (T, k) or route.counts.shape != (E,) or \
            route.tokens.shape != (1,):
        raise ValueError("route is not of these logits")
    for name, t, n in (("grad_weight", grad_weight, (T, k)), ("grad_loss", grad_loss, None)):
        if t is not None and (t.numel() != 1 if n is None else tuple(t.shape) != n):
            raise ValueError(f"{name} has shape {list(t.shape)}")
    dl, dp = c.result(out, (T, E), logits.dtype, "out", T * E)
    f32, i32 = torch.float32, torch.int32
    counts = route.counts
    cp, tp = c.ptr(counts, i32, "route.counts", E), c.ptr(route.tokens, i32, "route.tokens", 1)
    if tp != cp + 4 * E:   # a copy of what qmoe_route returned: the kernel reads both from one buffer
        counts = torch.cat((counts, route.tokens))
        cp = counts.data_ptr()
    c("qmoe_route_backward", logits.data_ptr(), _type(logits.dtype), ld, mp, T, E, k, int(renormalize),
      c.ptr(route.idx, i32, "route.idx", T * k), c.ptr(route.weight, f32, "route.weight", T * k),
      cp, c.opt(grad_weight, f32, "grad_weight", T * k),
      c.opt(grad_loss, f32, "grad_loss", 1), dp)
    return dl


def _slots(T: int, order):
    S = order.numel()
    if T < 1 or S < 1 or S % T:
        raise ValueError(f"order has {S} slots, not a multiple of {T} tokens")
    return S, S // T


def qmoe_gemm_f8(pool, P: int, xq, T: int, order, offsets, N: int, K: int, dtype=None, Y=None):
    """Y[slot][N] = expert's matrix times X[slot // k] for the slots of
    qmoe_route's order / offsets (k = order.numel() // T; T rows of X); slots
    without an expert get zeros."""
    torch = _torch()
    c, nb, na = _Call(pool, "pool"), qpacked_bytes_f8(N, K), qact_bytes_f8(T, K)
    _sizes("qmoe_gemm_f8", nb, na)
    S, k = _slots(T, order)
    dtype = dtype or (torch.float32 if Y is None else Y.dtype)
    code = _type(dtype)
    Y, yp = c.result(Y, (S, N), dtype, "Y", S * N)
    c("qmoe_gemm_f8", c.ptr(pool, torch.uint8, "pool", P * nb), P, c.ptr(xq, torch.uint8, "xq", na), T, k,
      c.ptr(order, torch.int32, "order", S), c.ptr(offsets, torch.int32, "offsets", P + 1),
      yp, code, N, K)
    return Y


def qmoe_gemm_f8_wgrad(dY, xq, T: int, order, offsets, P: int, N: int, K: int, dW=None, accumulate: bool = False):
    """dW[P][N][K] (fp32): for each expert, dY^T @ X over its slots (dY bf16 [slots][N], X packed with T rows)."""
    torch = _torch()
    c, na = _Call(dY, "dY"), qact_bytes_f8(T, K)
    _sizes("qmoe_gemm_f8_wgrad", na, qpacked_bytes_f8(N, K))
    S, k = _slots(T, order)
    if accumulate and dW is None:
        raise ValueError("accumulate needs dW")
    dW, wp = c.result(dW, (P, N, K), torch.float32, "dW", P * N * K)
    c("qmoe_gemm_f8_wgrad", c.ptr(dY, torch.bfloat16, "dY", S * N), c.ptr(xq, torch.uint8, "xq", na), T, k,
      c.ptr(order, torch.int32, "order", S), c.ptr(offsets, torch.int32, "offsets", P + 1), P,
      wp, int(accumulate), N, K)
    return dW


# --------------------------------------------------------------- measurement
def qg_set_gemv_shape(J: int = 0, R: int = 0, ksplit: int = 0, teams_per_wg: int = 0, teams: int = 0,
                      xl: int = -1, engine: int = -1, lanes: int = 0):
    lib().qg_set_gemv_shape(J, R, ksplit, teams_per_wg, teams, xl, engine, lanes)


def qg_read_probe(buf, sink, wgs: int, loads: int = 8, nbytes: int | None = None):
    """Streaming read of the uint8 device tensor `buf` (its first `nbytes`
    bytes, default all) by `wgs` workgroups with `loads` 16-byte loads in
    flight per lane (bandwidth probe)."""
    torch = _torch()
    n = buf.numel() if nbytes is None else int(nbytes)
    bp = _dev(buf, torch.uint8, "buf", n)
    sp = _dev(sink, torch.int32, "sink", wgs)
    _check("qg_read_probe", lib().qg_read_probe(bp, n, sp, wgs, loads, _stream()))


def qg_set_prefill_shape(splits: int = 0, bm: int = 0):
    lib().qg_set_prefill_shape(splits, bm)


def qg_device_cus(device: int = 0) -> int:
    n = ctypes.c_int(0)
    _check("qg_device_cus", lib().qg_device_cus(device, ctypes.byref(n)))
    return n.value


class KernelTimer:
    """HIP events recorded by the kernel launch itself (hipExtLaunchKernel),
    so elapsed() is the kernel's own execution time.  Uses the HIP runtime
    torch already loaded."""

    def __init__(self, count: int):
        self._hip = ctypes.CDLL("libamdhip64.so.7", mode=ctypes.RTLD_GLOBAL)
        self._hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        self._hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                                  ctypes.c_void_p]
        self._hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self._hip.hipEventSynchronize.argtypes = [ctypes.c_void_p]
        self.start = []
        self.stop = []
        for _ in range(count):
            a, b = ctypes.c_void_p(), ctypes.c_void_p()
            if self._hip.hipEventCreate(ctypes.byref(a)) or self._hip.hipEventCreate(ctypes.byref(b)):
                raise RuntimeError("hipEventCreate failed")
            self.start.append(a)
            self.stop.append(b)
        self.n = 0

    def arm(self):
        """The next library launch from this thread records into event pair n."""
        i = self.n
        lib().qg_time_next_launch(self.start[i], self.stop[i])
        self.n += 1

    def reset(self):
        self.n = 0

    def elapsed_ms(self) -> list[float]:
        out = []
        for i in range(self.n):
            self._hip.hipEventSynchronize(self.stop[i])
            ms = ctypes.c_float(0)
            rc = self._hip.hipEventElapsedTime(ctypes.byref(ms), self.start[i], self.stop[i])
            if rc != 0:
                raise RuntimeError(f"hipEventElapsedTime failed ({rc})")
            out.append(ms.value)
        return out

    def close(self):
        for e in self.start + self.stop:
            self._hip.hipEventDestroy(e)
        self.start, self.stop = [], []
