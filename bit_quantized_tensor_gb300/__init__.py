"""Python binding of libqgemm.so, the GB300 quantized tensor-core GEMM library.

Argument marshalling only: every step of every operation runs in the CUDA
kernels behind the C ABI declared in ``include/qgemm.h``.  PyTorch supplies
device memory and the current CUDA stream.  There is no fallback: if the
library is not built, or the tensors are not CUDA tensors, the calls raise.

Functions (same names as the C ABI):
  qgemm_s8(A, B)            exact int8 GEMM,  A: M x K int8, B: N x K int8 -> int32 M x N
  qgemm_s4(A, B, K)         exact int4 GEMM on packed operands (M x K/2, N x K/2 uint8)
  gemm_f16(A, B)            fp16 GEMM with fp32 accumulation -> fp16 M x N
  w4a16_gemm(X, Wq, Wscale) weight-only INT4 linear, per-group (128) fp16 scales
  w4a4_quantize(X, U)       per-row, per-64-block absmax INT4 quantizer (+ X.U)
  w4a4_gemm(...)            Y = (Q(X).Q(W)^T) (.) scale + (X.U).V + b
                            (alpha=...: the column-wise affine form,
                            Y = alpha (.) (...) + b, through w4a4_gemm_affine)
B / W operands are K-major (N x K row-major), the layout every call takes.

Microscaled 4-bit floating point (fmt "nv": blocks of 16 with e4m3 scales and a
tensor scale; "mx": blocks of 32 with power-of-two scales) and layer norm:
  fp4_tensor_scale(X)             the "nv" tensor scale of X
  fp4_quantize(X, fmt)            X -> packed operand (codes, scales)
  fp4_quantize_both(X, fmt)       packed operands of X and of its transpose
  fp4_dequantize(Xq, Xs, K, fmt)  the values of a packed operand
  fp4_gemm(Aq, As, Bq, Bs, K)     A . B^T (+ bias) of packed operands
  fp4_linear(X, Wq, Ws)           Q(X) . W^T (+ bias), X quantized in the call
  fp4_linear_backward(dY, X, ...) dX, dW and the bias gradient
  layer_norm(X, gamma, beta)      y, mean, rstd
  layer_norm_fp4(X, gamma, beta)  the same, y quantized to a packed operand
  layer_norm_backward(...)        dX, dgamma, dbeta
"""
from __future__ import annotations

import ctypes
import os
import re

from . import inputs  # noqa: F401  (seeded input generators)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemm.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "qgemm.h")

(QG_OK, QG_ERR_INVALID_ARG, QG_ERR_UNSUPPORTED, QG_ERR_MISALIGNED, QG_ERR_WORKSPACE, QG_ERR_CUDA,
 QG_ERR_TIMEOUT) = range(7)
STATUS_NAMES = {0: "QG_OK", 1: "QG_ERR_INVALID_ARG", 2: "QG_ERR_UNSUPPORTED",
                3: "QG_ERR_MISALIGNED", 4: "QG_ERR_WORKSPACE", 5: "QG_ERR_CUDA",
                6: "QG_ERR_TIMEOUT"}
QG_ROW_MAJOR, QG_COL_MAJOR = 0, 1
(QG_OP_S8, QG_OP_S4, QG_OP_F16, QG_OP_W4A16, QG_OP_W4A4, QG_OP_S8_HOST, QG_OP_W4A4_PREPACKED,
 QG_OP_W4A4_WEIGHTS, QG_OP_FP4_LINEAR, QG_OP_FP4_LINEAR_BACKWARD, QG_OP_LAYER_NORM_BACKWARD,
 QG_OP_FP4_TENSOR_SCALE) = range(12)
QG_FP4_NV, QG_FP4_MX = 0, 1
QG_F16, QG_BF16, QG_F32 = 0, 1, 2


class QgError(RuntimeError):
    def __init__(self, name: str, code: int):
        super().__init__(f"{name} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


class KernelBudgetC(ctypes.Structure):
    """qg_kernel_budget of the C ABI."""
    _fields_ = [("kernel", ctypes.c_char_p), ("threads", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("tmem_cols", ctypes.c_int), ("cluster", ctypes.c_int), ("min_ctas_per_sm", ctypes.c_int)]


_i64 = ctypes.c_int64
_p = ctypes.c_void_p
_sz = ctypes.c_size_t
_int = ctypes.c_int
_f32 = ctypes.c_float

# C signatures (restype, argtypes) of every exported function.
SIGNATURES = {
    "qg_status_string": (ctypes.c_char_p, [_int]),
    "qg_version": (_int, []),
    "qg_workspace_size": (_sz, [_int, _i64, _i64, _i64]),
    "qg_device_status": (_int, [_p]),
    "qg_device_status_detail": (_int, [ctypes.POINTER(ctypes.c_int), _p]),
    "qg_last_cuda_error": (_int, []),
    "qg_set_timeout_ns": (_int, [ctypes.c_uint64]),
    "qg_selftest_wait_timeout": (_int, [ctypes.c_uint64, _p]),
    "qg_selftest_deadlock": (_int, [_int, ctypes.c_uint64, _p]),
    "qg_kernel_budget_count": (_int, []),
    "qg_kernel_budget_get": (_int, [_int, ctypes.POINTER(KernelBudgetC)]),
    "qg_kernel_budget_measure": (_int, [_int, ctypes.POINTER(_int), ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "qg_set_s8_chunk": (_int, [_int]),
    "qg_set_gemm_path": (_int, [_int]),
    "qg_set_s4_path": (_int, [_int]),
    "qg_set_w4a4_pair_form": (_int, [_int]),
    "qg_set_l2_policy": (_int, [_int]),
    "qg_set_pdl": (_int, [_int]),
    "qg_set_w4a16_tc_form": (_int, [_int]),
    "qg_set_profile_events": (_int, [_p, _p]),
    "qgemm_s8": (_int, [_i64, _i64, _i64, _p, _i64, _int, _p, _i64, _int, _p, _i64, _p, _sz, _p]),
    "qgemm_s8_noalloc": (_int, [_i64, _i64, _i64, _p, _i64, _int, _p, _i64, _int, _p, _i64, _p]),
    "qgemm_s8_host": (_int, [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _sz, _p]),
    "qgemm_s4": (_int, [_i64, _i64, _i64, _p, _i64, _int, _p, _i64, _int, _p, _i64, _p, _sz, _p]),
    "gemm_f16": (_int, [_i64, _i64, _i64, _p, _i64, _int, _p, _i64, _int, _p, _i64, _p]),
    "w4a16_gemm": (_int, [_i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _i64, _p]),
    "w4a4_quantize": (_int, [_i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _p]),
    "w4a4_gemm": (_int, [_i64, _i64, _i64, _p, _p, _p, _p, _i64, _p, _p, _i64, _p, _p, _i64,
                         _p, _sz, _p]),
    "w4a4_gemm_affine": (_int, [_i64, _i64, _i64, _p, _p, _p, _p, _i64, _p, _p, _i64, _p, _p, _p,
                                _i64, _p, _sz, _p]),
    "w4a4_prepack_weights": (_int, [_i64, _i64, _p, _p, _i64, _p, _p, _sz, _p]),
    "w4a4_gemm_prepacked": (_int, [_i64, _i64, _i64, _p, _p, _p, _sz, _i64, _p, _p, _i64, _p, _p, _i64,
                                   _p, _sz, _p]),
    "qg_block_kernel_budget_count": (_int, []),
    "qg_block_kernel_budget_get": (_int, [_int, ctypes.POINTER(KernelBudgetC)]),
    "qg_block_kernel_budget_measure": (_int, [_int, ctypes.POINTER(_int), ctypes.POINTER(_int),
                                              ctypes.POINTER(_int)]),
    "qg_set_fp4_path": (_int, [_int, _int]),
    "qg_fp4_codes_ld": (_i64, [_i64]),
    "qg_fp4_scale_bytes": (_sz, [_int, _i64, _i64]),
    "fp4_tensor_scale": (_int, [_int, _i64, _i64, _p, _i64, _p, _p, _sz, _p]),
    "fp4_quantize": (_int, [_int, _int, _i64, _i64, _p, _i64, _p, _p, _p, _p]),
    "fp4_quantize_both": (_int, [_int, _int, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p, _p]),
    "fp4_dequantize": (_int, [_int, _int, _i64, _i64, _p, _p, _p, _p, _i64, _p]),
    "fp4_gemm": (_int, [_int, _int, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p]),
    "fp4_linear": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _i64, _p, _sz,
                          _p]),
    "fp4_linear_backward": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _p, _p, _p,
                                   _p, _i64, _p, _i64, _p, _p, _sz, _p]),
    "layer_norm": (_int, [_int, _i64, _i64, _p, _i64, _p, _p, _int, _f32, _p, _i64, _p, _p, _p]),
    "layer_norm_fp4": (_int, [_int, _int, _i64, _i64, _p, _i64, _p, _p, _int, _f32, _p, _p, _p, _p, _p,
                              _p]),
    "layer_norm_backward": (_int, [_int, _i64, _i64, _p, _i64, _p, _i64, _p, _int, _p, _p, _p, _i64, _p,
                                   _p, _p, _sz, _p]),
}

_lib = None


def header_functions() -> list[str]:
    """Names of the functions include/qgemm.h declares."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", txt, flags=re.M)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                f"g.build()\"` (needs nvcc); there is no fallback implementation")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:  # an import statement on every call costs more than the call
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream=None) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check(name: str, code: int) -> None:
    if code != QG_OK:
        err = QgError(name, code)
        if code == 5:  # QG_ERR_CUDA: attach the failing CUDA call's code
            err.cuda_error = int(lib().qg_last_cuda_error())
            err.args = (f"{err.args[0]} (CUDA error code {err.cuda_error})",)
        raise err


def _cuda(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() >= 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t


def workspace_size(op: int, M: int, N: int, K: int) -> int:
    return int(lib().qg_workspace_size(op, M, N, K))


def _workspace(op, M, N, K, device, ws):
    torch = _torch()
    need = workspace_size(op, M, N, K)
    if ws is None:
        # torch's caching allocator returns blocks aligned to at least 512 bytes
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def device_status(stream=None) -> int:
    return int(lib().qg_device_status(_stream(stream)))


STATUS_WORDS = ("code", "site", "count", "block", "parity", "barrier")


def device_status_detail(stream=None) -> dict:
    """Reads and clears the device status word; returns its six fields by name
    ("code" is QG_OK when no wait ran out since the last read)."""
    words = (ctypes.c_int * len(STATUS_WORDS))()
    code = int(lib().qg_device_status_detail(words, _stream(stream)))
    if code == QG_ERR_CUDA:
        raise QgError("qg_device_status_detail", code)
    return dict(zip(STATUS_WORDS, (int(w) for w in words)))


def kernel_budgets(measure: bool = False, table: str = "gemm") -> list:
    """One of the library's kernel budget tables, one dict per kernel instance:
    table "gemm" (the GEMMs and their quantizers) or "block" (microscaled 4-bit
    operators and layer norm).  With measure=True (needs a device) each entry
    also gets the compiled kernel's registers per thread, static shared memory
    and the CTAs per SM the device's occupancy calculator gives at the entry's
    launch shape."""
    if table not in ("gemm", "block"):
        raise ValueError("table must be 'gemm' or 'block'")
    stem = "qg_kernel_budget" if table == "gemm" else "qg_block_kernel_budget"
    L = lib()
    out = []
    for i in range(int(getattr(L, f"{stem}_count")())):
        b = KernelBudgetC()
        _check(f"{stem}_get", getattr(L, f"{stem}_get")(i, ctypes.byref(b)))
        e = {name: getattr(b, name) for name, _ in KernelBudgetC._fields_}
        e["kernel"] = b.kernel.decode()
        if measure:
            regs, ssm, ctas = _int(), _int(), _int()
            _check(f"{stem}_measure", getattr(L, f"{stem}_measure")(
                i, ctypes.byref(regs), ctypes.byref(ssm), ctypes.byref(ctas)))
            e.update(regs_per_thread=regs.value, static_smem_bytes=ssm.value, ctas_per_sm=ctas.value)
        out.append(e)
    return out


def set_timeout_ns(ns: int) -> None:
    _check("qg_set_timeout_ns", lib().qg_set_timeout_ns(int(ns)))


def qgemm_s8(A, B, C=None, ws=None, stream=None):
    torch = _torch()
    _cuda(A, torch.int8, "A")
    _cuda(B, torch.int8, "B")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("B must be N x K (K-major)")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, device=A.device)
    _cuda(C, torch.int32, "C")
    ws, wsb = _workspace(QG_OP_S8, M, N, K, A.device, ws)
    _check("qgemm_s8", lib().qgemm_s8(M, N, K, A.data_ptr(), A.stride(0), QG_ROW_MAJOR,
                                      B.data_ptr(), B.stride(0), QG_COL_MAJOR,
                                      C.data_ptr(), C.stride(0), ws.data_ptr(), wsb,
                                      _stream(stream)))
    return C


def _host(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise TypeError(f"{name} must be a CPU (host) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")


def qgemm_s8_host(A, B, C=None, ws=None, stream=None):
    """qgemm_s8 with A (M x K int8), B (N x K int8) and C (M x N int32) in host
    memory; the copies both ways run inside the call, overlapped with the
    arithmetic.  Use page-locked tensors (``pin_memory()``) for full link
    speed.  The call is asynchronous: C is complete once ``stream`` (default:
    the current stream) has been synchronized.  ``ws`` is a device workspace
    (allocated on the current device when None)."""
    torch = _torch()
    _host(A, torch.int8, "A")
    _host(B, torch.int8, "B")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("B must be N x K (K-major)")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, pin_memory=A.is_pinned())
    _host(C, torch.int32, "C")
    ws, wsb = _workspace(QG_OP_S8_HOST, M, N, K, torch.device("cuda", torch.cuda.current_device()), ws)
    _check("qgemm_s8_host", lib().qgemm_s8_host(M, N, K, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0),
                                                C.data_ptr(), C.stride(0), ws.data_ptr(), wsb,
                                                _stream(stream)))
    return C


def qgemm_s4(A, B, K: int, C=None, ws=None, stream=None):
    torch = _torch()
    _cuda(A, torch.uint8, "A")
    _cuda(B, torch.uint8, "B")
    M, N = A.shape[0], B.shape[0]
    if A.shape[1] * 2 < K or B.shape[1] * 2 < K:
        raise ValueError("packed operands must hold K/2 bytes per row")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, device=A.device)
    _cuda(C, torch.int32, "C")
    ws, wsb = _workspace(QG_OP_S4, M, N, K, A.device, ws)
    _check("qgemm_s4", lib().qgemm_s4(M, N, K, A.data_ptr(), A.stride(0), QG_ROW_MAJOR,
                                      B.data_ptr(), B.stride(0), QG_COL_MAJOR,
                                      C.data_ptr(), C.stride(0), ws.data_ptr(), wsb,
                                      _stream(stream)))
    return C


def gemm_f16(A, B, C=None, stream=None):
    torch = _torch()
    _cuda(A, torch.float16, "A")
    _cuda(B, torch.float16, "B")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("B must be N x K (K-major)")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _cuda(C, torch.float16, "C")
    _check("gemm_f16", lib().gemm_f16(M, N, K, A.data_ptr(), A.stride(0), QG_ROW_MAJOR,
                                      B.data_ptr(), B.stride(0), QG_COL_MAJOR,
                                      C.data_ptr(), C.stride(0), _stream(stream)))
    return C


def w4a16_gemm(X, Wq, Wscale, group: int = 128, Y=None, stream=None):
    torch = _torch()
    _cuda(X, torch.float16, "X")
    _cuda(Wq, torch.uint8, "Wq")
    _cuda(Wscale, torch.float16, "Wscale")
    M, K = X.shape
    N = Wq.shape[0]
    if not (Wq.is_contiguous() and Wscale.is_contiguous()):
        raise ValueError("Wq and Wscale must be contiguous")
    if Wq.shape[1] * 2 != K or tuple(Wscale.shape) != (N, K // group):
        raise ValueError("Wq must be N x K/2 bytes and Wscale N x K/group")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _cuda(Y, torch.float16, "Y")
    _check("w4a16_gemm", lib().w4a16_gemm(M, N, K, X.data_ptr(), X.stride(0), Wq.data_ptr(),
                                          Wscale.data_ptr(), group, Y.data_ptr(), Y.stride(0),
                                          _stream(stream)))
    return Y


def w4a4_quantize(X, Ut=None, block: int = 64, out=None, stream=None):
    """Returns (Xq M x K/2 uint8, Xscale M x K/block fp16, XU M x rank fp16 or None).

    Ut is the low-rank down-projection transposed (rank x K fp16, the weight
    of a K -> rank linear layer); XU = X . Ut^T.
    """
    torch = _torch()
    _cuda(X, torch.float32, "X")
    M, K = X.shape
    rank = 0
    U = Ut
    if U is not None:
        _cuda(U, torch.float16, "Ut")
        if not U.is_contiguous() or U.dim() != 2 or U.shape[1] != K:
            raise ValueError("Ut must be a contiguous rank x K fp16 matrix")
        rank = U.shape[0]
    if out is None:
        Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device)
        Xs = torch.empty((M, K // block), dtype=torch.float16, device=X.device)
        XU = torch.empty((M, rank), dtype=torch.float16, device=X.device) if rank else None
    else:
        Xq, Xs, XU = out
    _check("w4a4_quantize", lib().w4a4_quantize(
        M, K, X.data_ptr(), X.stride(0), U.data_ptr() if rank else None, rank,
        Xq.data_ptr(), Xs.data_ptr(), XU.data_ptr() if rank else None, block, _stream(stream)))
    return Xq, Xs, XU


def w4a4_gemm(Xq, Xscale, Wq, Wscale, K: int, XU=None, Vt=None, bias=None, block: int = 64,
              Y=None, ws=None, stream=None, alpha=None):
    """Y = (Q(X).Q(W)^T) (.) scale + XU . Vt^T + bias, fp16 M x N.

    Vt is the low-rank up-projection transposed (N x rank fp16, the weight of
    a rank -> N linear layer).  With alpha (N fp16 column multipliers) the
    call is w4a4_gemm_affine: Y = alpha (.) ((...) (.) scale + XU . Vt^T) + bias.
    """
    torch = _torch()
    V = Vt
    _cuda(Xq, torch.uint8, "Xq")
    _cuda(Wq, torch.uint8, "Wq")
    _cuda(Xscale, torch.float16, "Xscale")
    _cuda(Wscale, torch.float16, "Wscale")
    M, N = Xq.shape[0], Wq.shape[0]
    rank = 0
    if XU is not None:
        _cuda(XU, torch.float16, "XU")
        _cuda(V, torch.float16, "Vt")
        rank = XU.shape[1]
        if not V.is_contiguous() or V.dim() != 2 or V.shape != (N, rank):
            raise ValueError("Vt must be a contiguous N x rank fp16 matrix")
    if bias is not None:
        _cuda(bias, torch.float16, "bias")
    if alpha is not None:
        _cuda(alpha, torch.float16, "alpha")
        if alpha.numel() != N:
            raise ValueError("alpha must hold N fp16 column multipliers")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=Xq.device)
    _cuda(Y, torch.float16, "Y")
    ws, wsb = _workspace(QG_OP_W4A4, M, N, K, Xq.device, ws)
    head = (M, N, K, Xq.data_ptr(), Xscale.data_ptr(), Wq.data_ptr(), Wscale.data_ptr(), block,
            XU.data_ptr() if rank else None, V.data_ptr() if rank else None, rank)
    tail = (bias.data_ptr() if bias is not None else None, Y.data_ptr(), Y.stride(0),
            ws.data_ptr(), wsb, _stream(stream))
    if alpha is None:
        _check("w4a4_gemm", lib().w4a4_gemm(*head, *tail))
    else:
        _check("w4a4_gemm_affine", lib().w4a4_gemm_affine(*head, alpha.data_ptr(), *tail))
    return Y


def w4a4_prepack_weights(Wq, Wscale, K: int, alpha=None, block: int = 64, out=None, stream=None):
    """The weight side of w4a4_gemm prepared once: a uint8 device buffer for
    w4a4_gemm_prepacked (with the column multiplier alpha folded in, if given)."""
    torch = _torch()
    _cuda(Wq, torch.uint8, "Wq")
    _cuda(Wscale, torch.float16, "Wscale")
    N = Wq.shape[0]
    if alpha is not None:
        _cuda(alpha, torch.float16, "alpha")
        if alpha.numel() != N:
            raise ValueError("alpha must hold N fp16 column multipliers")
    nbytes = workspace_size(QG_OP_W4A4_WEIGHTS, 1, N, K)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=Wq.device)
    _check("w4a4_prepack_weights", lib().w4a4_prepack_weights(
        N, K, Wq.data_ptr(), Wscale.data_ptr(), block,
        alpha.data_ptr() if alpha is not None else None, out.data_ptr(), out.numel(), _stream(stream)))
    return out


def w4a4_gemm_prepacked(Xq, Xscale, packed, N: int, K: int, XU=None, Vt=None, bias=None, block: int = 64,
                        Y=None, ws=None, stream=None):
    """w4a4_gemm with weights from w4a4_prepack_weights (only X is converted per call)."""
    torch = _torch()
    _cuda(Xq, torch.uint8, "Xq")
    _cuda(Xscale, torch.float16, "Xscale")
    _cuda(packed, torch.uint8, "packed")
    M = Xq.shape[0]
    rank = 0
    V = Vt
    if XU is not None:
        _cuda(XU, torch.float16, "XU")
        _cuda(V, torch.float16, "Vt")
        rank = XU.shape[1]
        if not V.is_contiguous() or V.dim() != 2 or V.shape != (N, rank):
            raise ValueError("Vt must be a contiguous N x rank fp16 matrix")
    if bias is not None:
        _cuda(bias, torch.float16, "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=Xq.device)
    _cuda(Y, torch.float16, "Y")
    ws, wsb = _workspace(QG_OP_W4A4_PREPACKED, M, N, K, Xq.device, ws)
    _check("w4a4_gemm_prepacked", lib().w4a4_gemm_prepacked(
        M, N, K, Xq.data_ptr(), Xscale.data_ptr(), packed.data_ptr(), packed.numel(), block,
        XU.data_ptr() if rank else None, V.data_ptr() if rank else None, rank,
        bias.data_ptr() if bias is not None else None, Y.data_ptr(), Y.stride(0),
        ws.data_ptr(), wsb, _stream(stream)))
    return Y


# ---------------------------------------------------------------- microscaled 4-bit, layer norm
#
# A small call takes a few microseconds on the device, so the host side counts:
# the ordinary call goes through _ordinary(); for the others each operand is looked
# at once, and the current stream comes as a raw handle (the stream object that
# torch.cuda.current_stream() builds costs 3 us).
#
# A call with stream= is the same call with that stream as the current one: what it
# allocates (outputs, workspaces) comes from that stream's pool, whose blocks nothing
# on another stream may still use.

_host_module = None
_HOST_ENTRIES = ("qg_workspace_size", "fp4_tensor_scale", "fp4_quantize", "fp4_dequantize", "fp4_gemm", "fp4_linear",
                 "fp4_linear_backward", "layer_norm", "layer_norm_fp4", "layer_norm_backward")


class _NotBuilt:
    """Stands for the module where there is none: no call is ordinary."""

    def __getattr__(self, name):
        return lambda *args: None


def _ordinary():
    """csrc/qg_host.cpp: the ordinary call of each function below, in C++.  Its functions
    return None for any other call, which then goes through ctypes, as all do where the
    module was not built or is another torch's."""
    global _host_module
    if _host_module is None:
        _torch()
        L = lib()
        try:
            from . import _qg_host
        except ImportError as e:
            import warnings
            warnings.warn(f"_qg_host.so is missing or does not load ({e}): small calls take longer.  Build it with "
                          f"`python -c \"import __graft_entry__ as g; g.build()\"`", RuntimeWarning, stacklevel=3)
            _host_module = _NotBuilt()
            return _host_module
        _qg_host.bind([ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _HOST_ENTRIES])
        _host_module = _qg_host
    return _host_module


_dtype_ids = None


def _dtype_id(dtype, name):
    global _dtype_ids
    if _dtype_ids is None:
        torch = _torch()
        _dtype_ids = {torch.float16: QG_F16, torch.bfloat16: QG_BF16, torch.float32: QG_F32}
    i = _dtype_ids.get(dtype)
    if i is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {dtype}")
    return i


def _fmt_id(fmt):
    if fmt == "nv":
        return QG_FP4_NV
    if fmt == "mx":
        return QG_FP4_MX
    raise ValueError(f"fmt must be 'nv' or 'mx', got {fmt!r}")


def _raw_stream(device):
    return _torch_module._C._cuda_getCurrentRawStream(device.index)


def _on(t, name, device):
    if not isinstance(t, _torch_module.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if device is None:  # the first operand: the library launches on the current device
        if t.device.index != _torch_module.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_torch_module.cuda.current_device()}")
    elif t.device != device:
        raise ValueError(f"{name} is on {t.device}, other operands on {device}")


def _matrix(t, name, device=None, dtype=None, rows=None, cols=None):
    """Checks a 2-D matrix with unit column stride; returns its leading dimension."""
    _on(t, name, device)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    m, k = shape
    if rows is not None and (m != rows or k != cols):
        raise ValueError(f"{name} must be {rows} x {cols}, got {m} x {k}")
    ld, unit = t.stride()
    if unit != 1 and k > 1 and m > 0:
        raise ValueError(f"{name} must have a contiguous last dimension")
    if m <= 1:
        return k
    if ld < k:
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _packed_shapes(rows, K, fmt):
    per_tile = 64 if fmt == "nv" else 128  # values along K that a scale tile covers
    return (rows, (K + 31) // 32 * 16), ((rows + 127) // 128, (K + per_tile - 1) // per_tile, 512)


def _packed(codes, scales, name, fmt, K, device=None):
    """Checks a packed operand; returns its number of rows."""
    u8 = _torch_module.uint8
    _on(codes, name, device)
    _on(scales, name, codes.device)
    if (codes.dtype is not u8 or scales.dtype is not u8 or not codes.is_contiguous()
            or not scales.is_contiguous()):
        raise TypeError(f"{name}: codes and scales must be contiguous uint8")
    shape = codes.shape
    rows = shape[0] if len(shape) == 2 else 0
    want, (tr, tc, _) = _packed_shapes(rows, K, fmt)
    if shape != want:
        raise ValueError(f"{name}: codes must be rows x {want[1]} bytes for K = {K}")
    if scales.numel() != tr * tc * 512:
        raise ValueError(f"{name}: scales do not match {rows} rows of {K} values in format {fmt!r}")
    return rows


def _new_packed(rows, K, fmt, device):
    torch = _torch_module
    c, s = _packed_shapes(rows, K, fmt)
    return torch.empty(c, dtype=torch.uint8, device=device), torch.empty(s, dtype=torch.uint8, device=device)


def _one_f32(t, name, fmt, device):
    """Address of a tensor scale (one fp32 on the device), or None."""
    if t is None:
        return None
    if fmt == "mx":
        raise ValueError(f"{name}: format 'mx' has no tensor scale")
    _on(t, name, device)
    if t.dtype is not _torch_module.float32 or t.numel() != 1:
        raise TypeError(f"{name} must be one float32")
    return t.data_ptr()


def _vector(t, name, n, dtype, device):
    """Address of a contiguous vector of n values, or None."""
    if t is None:
        return None
    _on(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values")
    return t.data_ptr()


def _scratch(ws, need, device):
    """Address and size of the caller's workspace, or of a new one of the current stream."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = _torch_module.empty(need, dtype=_torch_module.uint8, device=device)
    else:
        _on(ws, "ws", device)
        need = ws.numel() * ws.element_size()
    return ws, ws.data_ptr(), need


def _weights(gamma, beta, D, xdtype, device):
    """Addresses of gamma and beta and the id of their common type (that of X, or fp32)."""
    w = gamma if gamma is not None else beta
    if w is None:
        return None, None, _dtype_id(xdtype, "X")
    _on(w, "gamma", device)
    wdtype = w.dtype
    if wdtype is not xdtype and wdtype is not _torch_module.float32:
        raise TypeError(f"gamma and beta must be {xdtype} or float32, got {wdtype}")
    if gamma is not None and beta is not None and beta.dtype is not wdtype:
        raise TypeError("gamma and beta must have the same type")
    return (_vector(gamma, "gamma", D, wdtype, device), _vector(beta, "beta", D, wdtype, device),
            _dtype_id(wdtype, "gamma"))


def fp4_tensor_scale(X, out=None, ws=None, stream=None):
    """The "nv" tensor scale of X: max(|x|) / 2688 over its finite values, one fp32 on the device."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_tensor_scale(X, out, ws)
    if out is None and ws is None:
        scale = _ordinary().fp4_tensor_scale(X)
        if scale is not None:
            return scale
    torch = _torch()
    ld = _matrix(X, "X")
    dev = X.device
    dt = _dtype_id(X.dtype, "X")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=dev)
    ptr = _one_f32(out, "out", "nv", dev)
    ws, wsp, wsb = _scratch(ws, 4096, dev)
    M, K = X.shape
    _check("fp4_tensor_scale", lib().fp4_tensor_scale(dt, M, K, X.data_ptr(), ld, ptr, wsp, wsb,
                                                      _raw_stream(dev)))
    return out


def fp4_quantize(X, fmt: str = "nv", scale=None, out=None, stream=None):
    """X (M x K) -> (codes, scales), blocks along its rows; scale: the "nv" tensor scale (None = 1)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_quantize(X, fmt, scale, out)
    if out is None:
        both = _ordinary().fp4_quantize(X, fmt, scale)
        if both is not None:
            return both
    _torch()
    f = _fmt_id(fmt)
    ld = _matrix(X, "X")
    dev = X.device
    dt = _dtype_id(X.dtype, "X")
    M, K = X.shape
    if out is None:
        Xq, Xs = _new_packed(M, K, fmt, dev)
    else:
        Xq, Xs = out
        if _packed(Xq, Xs, "out", fmt, K, dev) != M:
            raise ValueError(f"out must have {M} rows")
    _check("fp4_quantize", lib().fp4_quantize(
        f, dt, M, K, X.data_ptr(), ld, _one_f32(scale, "scale", fmt, dev), Xq.data_ptr(), Xs.data_ptr(),
        _raw_stream(dev)))
    return Xq, Xs


def fp4_quantize_both(X, fmt: str = "nv", scale=None, out=None, stream=None):
    """X (M x K) -> (codes, scales) of X and (codes, scales) of its transpose, reading X once."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_quantize_both(X, fmt, scale, out)
    _torch()
    f = _fmt_id(fmt)
    ld = _matrix(X, "X")
    dev = X.device
    dt = _dtype_id(X.dtype, "X")
    M, K = X.shape
    if out is None:
        out = _new_packed(M, K, fmt, dev) + _new_packed(K, M, fmt, dev)
    elif (_packed(out[0], out[1], "out", fmt, K, dev) != M
          or _packed(out[2], out[3], "transposed out", fmt, M, dev) != K):
        raise ValueError(f"out must have {M} rows, and {K} transposed")
    Xq, Xs, Tq, Ts = out
    _check("fp4_quantize_both", lib().fp4_quantize_both(
        f, dt, M, K, X.data_ptr(), ld, _one_f32(scale, "scale", fmt, dev), Xq.data_ptr(), Xs.data_ptr(),
        Tq.data_ptr(), Ts.data_ptr(), _raw_stream(dev)))
    return Xq, Xs, Tq, Ts


def fp4_dequantize(Xq, Xs, K: int, fmt: str = "nv", scale=None, dtype=None, Y=None, stream=None):
    """The values (M x K) of a packed operand, in `dtype` (default: that of Y, or float32)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_dequantize(Xq, Xs, K, fmt, scale, dtype, Y)
    if Y is None:
        values = _ordinary().fp4_dequantize(Xq, Xs, K, fmt, scale, dtype)
        if values is not None:
            return values
    torch = _torch()
    f = _fmt_id(fmt)
    M = _packed(Xq, Xs, "X", fmt, K)
    dev = Xq.device
    if Y is None:
        Y = torch.empty((M, K), dtype=dtype or torch.float32, device=dev)
        ld = K
    else:
        ld = _matrix(Y, "Y", dev, dtype, M, K)
    _check("fp4_dequantize", lib().fp4_dequantize(
        f, _dtype_id(Y.dtype, "Y"), M, K, Xq.data_ptr(), Xs.data_ptr(), _one_f32(scale, "scale", fmt, dev),
        Y.data_ptr(), ld, _raw_stream(dev)))
    return Y


def fp4_gemm(Aq, As, Bq, Bs, K: int, fmt: str = "nv", a_scale=None, b_scale=None, bias=None, dtype=None,
             Y=None, stream=None):
    """Y = A . B^T + bias of packed A (M x K) and B (N x K), in `dtype` (default: that of Y, or bfloat16)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_gemm(Aq, As, Bq, Bs, K, fmt, a_scale, b_scale, bias, dtype, Y)
    if Y is None:
        product = _ordinary().fp4_gemm(Aq, As, Bq, Bs, K, fmt, a_scale, b_scale, bias, dtype)
        if product is not None:
            return product
    torch = _torch()
    f = _fmt_id(fmt)
    M = _packed(Aq, As, "A", fmt, K)
    dev = Aq.device
    N = _packed(Bq, Bs, "B", fmt, K, dev)
    if Y is None:
        dtype = dtype or torch.bfloat16
        dt = _dtype_id(dtype, "Y")
        Y = torch.empty((M, N), dtype=dtype, device=dev)
        ld = N
    else:
        ld = _matrix(Y, "Y", dev, dtype, M, N)
        dtype = Y.dtype
        dt = _dtype_id(dtype, "Y")
    _check("fp4_gemm", lib().fp4_gemm(
        f, dt, M, N, K, Aq.data_ptr(), As.data_ptr(), _one_f32(a_scale, "a_scale", fmt, dev), Bq.data_ptr(),
        Bs.data_ptr(), _one_f32(b_scale, "b_scale", fmt, dev), _vector(bias, "bias", N, dtype, dev), Y.data_ptr(),
        ld, _raw_stream(dev)))
    return Y


def fp4_linear(X, Wq, Ws, fmt: str = "nv", x_scale=None, w_scale=None, bias=None, Y=None, ws=None, stream=None):
    """Y = Q(X) . W^T + bias with packed weights W (N x K); X (M x K) is quantized in the call, Y has its type."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_linear(X, Wq, Ws, fmt, x_scale, w_scale, bias, Y, ws)
    if Y is None and ws is None:
        product = _ordinary().fp4_linear(X, Wq, Ws, fmt, x_scale, w_scale, bias)
        if product is not None:
            return product
    torch = _torch()
    f = _fmt_id(fmt)
    ldx = _matrix(X, "X")
    dev = X.device
    dtype = X.dtype
    dt = _dtype_id(dtype, "X")
    M, K = X.shape
    N = _packed(Wq, Ws, "W", fmt, K, dev)
    if Y is None:
        Y = torch.empty((M, N), dtype=dtype, device=dev)
        ldy = N
    else:
        ldy = _matrix(Y, "Y", dev, dtype, M, N)
    L = lib()
    ws, wsp, wsb = _scratch(ws, L.qg_workspace_size(QG_OP_FP4_LINEAR, M, N, K), dev)
    _check("fp4_linear", L.fp4_linear(
        f, dt, M, N, K, X.data_ptr(), ldx, _one_f32(x_scale, "x_scale", fmt, dev), Wq.data_ptr(), Ws.data_ptr(),
        _one_f32(w_scale, "w_scale", fmt, dev), _vector(bias, "bias", N, dtype, dev), Y.data_ptr(), ldy,
        wsp, wsb, _raw_stream(dev)))
    return Y


def fp4_linear_backward(dY, X, Wtq, Wts, fmt: str = "nv", dy_scale=None, x_scale=None, w_scale=None,
                        need_dx: bool = True, need_dw: bool = True, need_db: bool = True, out=None, ws=None,
                        stream=None):
    """Gradients (dX, dW, db) of Y = X . W^T + bias from quantized products.

    Wtq, Wts: the packed transpose of W (K rows, blocks along N; the last two
    results of fp4_quantize_both(W)).  dX and dW have the type of dY, db (the
    column sums of dY) is fp32.  A gradient that is not needed is None.
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return fp4_linear_backward(dY, X, Wtq, Wts, fmt, dy_scale, x_scale, w_scale, need_dx, need_dw, need_db, out, ws)
    if need_dx and need_dw and need_db and out is None and ws is None:
        grads = _ordinary().fp4_linear_backward(dY, X, Wtq, Wts, fmt, dy_scale, x_scale, w_scale)
        if grads is not None:
            return grads
    torch = _torch()
    f = _fmt_id(fmt)
    lddy = _matrix(dY, "dY")
    dev, dtype = dY.device, dY.dtype
    dt = _dtype_id(dtype, "dY")
    M, N = dY.shape
    _on(X, "X", dev)
    K = X.shape[-1]
    ldx = _matrix(X, "X", dev, dtype, M, K)
    if _packed(Wtq, Wts, "W^T", fmt, N, dev) != K:
        raise ValueError(f"W^T must have {K} rows")
    if out is None:
        out = (torch.empty((M, K), dtype=dtype, device=dev) if need_dx else None,
               torch.empty((N, K), dtype=dtype, device=dev) if need_dw else None,
               torch.empty(N, dtype=torch.float32, device=dev) if need_db else None)
    dX, dW, db = out
    lddx = 0 if dX is None else _matrix(dX, "dX", dev, dtype, M, K)
    lddw = 0 if dW is None else _matrix(dW, "dW", dev, dtype, N, K)
    if dX is None and dW is None and db is None:
        return out
    L = lib()
    ws, wsp, wsb = _scratch(ws, L.qg_workspace_size(QG_OP_FP4_LINEAR_BACKWARD, M, N, K), dev)
    _check("fp4_linear_backward", L.fp4_linear_backward(
        f, dt, M, N, K, dY.data_ptr(), lddy, _one_f32(dy_scale, "dy_scale", fmt, dev), X.data_ptr(), ldx,
        _one_f32(x_scale, "x_scale", fmt, dev), Wtq.data_ptr(), Wts.data_ptr(),
        _one_f32(w_scale, "w_scale", fmt, dev), None if dX is None else dX.data_ptr(), lddx,
        None if dW is None else dW.data_ptr(), lddw, _vector(db, "db", N, torch.float32, dev),
        wsp, wsb, _raw_stream(dev)))
    return out


def _stats(stats, M, device):
    """mean and rstd: the caller's (checked) or new ones."""
    torch = _torch_module
    f32 = torch.float32
    if stats is None:
        return torch.empty(M, dtype=f32, device=device), torch.empty(M, dtype=f32, device=device)
    mean, rstd = stats
    _vector(mean, "mean", M, f32, device)
    _vector(rstd, "rstd", M, f32, device)
    return mean, rstd


def layer_norm(X, gamma=None, beta=None, eps: float = 1e-5, Y=None, stats=None, stream=None):
    """(Y, mean, rstd) of the rows of X (M x D); gamma and beta in X's type or fp32 (None = 1, 0)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return layer_norm(X, gamma, beta, eps, Y, stats)
    if Y is None and stats is None:
        result = _ordinary().layer_norm(X, gamma, beta, eps)
        if result is not None:
            return result
    torch = _torch()
    ldx = _matrix(X, "X")
    dev, dtype = X.device, X.dtype
    dt = _dtype_id(dtype, "X")
    M, D = X.shape
    g, b, wd = _weights(gamma, beta, D, dtype, dev)
    if Y is None:
        Y = torch.empty((M, D), dtype=dtype, device=dev)
        ldy = D
    else:
        ldy = _matrix(Y, "Y", dev, dtype, M, D)
    mean, rstd = _stats(stats, M, dev)
    _check("layer_norm", lib().layer_norm(dt, M, D, X.data_ptr(), ldx, g, b, wd, eps, Y.data_ptr(), ldy,
                                          mean.data_ptr(), rstd.data_ptr(), _raw_stream(dev)))
    return Y, mean, rstd


def layer_norm_fp4(X, gamma=None, beta=None, eps: float = 1e-5, fmt: str = "nv", scale=None, out=None, stats=None,
                   stream=None):
    """(codes, scales, mean, rstd): layer_norm of X with y quantized instead of stored.

    mean and rstd are None unless stats is True (new ones) or gives the two tensors.
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return layer_norm_fp4(X, gamma, beta, eps, fmt, scale, out, stats)
    if out is None and (stats is None or stats is True):
        result = _ordinary().layer_norm_fp4(X, gamma, beta, eps, fmt, scale, stats is True)
        if result is not None:
            return result
    _torch()
    f = _fmt_id(fmt)
    ldx = _matrix(X, "X")
    dev, dtype = X.device, X.dtype
    dt = _dtype_id(dtype, "X")
    M, D = X.shape
    g, b, wd = _weights(gamma, beta, D, dtype, dev)
    if out is None:
        Xq, Xs = _new_packed(M, D, fmt, dev)
    else:
        Xq, Xs = out
        if _packed(Xq, Xs, "out", fmt, D, dev) != M:
            raise ValueError(f"out must have {M} rows")
    mean, rstd = (None, None) if stats is None else _stats(None if stats is True else stats, M, dev)
    _check("layer_norm_fp4", lib().layer_norm_fp4(
        f, dt, M, D, X.data_ptr(), ldx, g, b, wd, eps, _one_f32(scale, "scale", fmt, dev), Xq.data_ptr(),
        Xs.data_ptr(), None if mean is None else mean.data_ptr(), None if rstd is None else rstd.data_ptr(),
        _raw_stream(dev)))
    return Xq, Xs, mean, rstd


def layer_norm_backward(dY, X, gamma, mean, rstd, out=None, ws=None, stream=None):
    """(dX, dgamma, dbeta) of layer_norm, with the mean and rstd it returned; dgamma and dbeta are fp32."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return layer_norm_backward(dY, X, gamma, mean, rstd, out, ws)
    if out is None and ws is None:
        grads = _ordinary().layer_norm_backward(dY, X, gamma, mean, rstd)
        if grads is not None:
            return grads
    torch = _torch()
    ldx = _matrix(X, "X")
    dev, dtype, f32 = X.device, X.dtype, torch.float32
    dt = _dtype_id(dtype, "X")
    M, D = X.shape
    lddy = _matrix(dY, "dY", dev, dtype, M, D)
    g, _, wd = _weights(gamma, None, D, dtype, dev)
    if out is None:
        dX = torch.empty((M, D), dtype=dtype, device=dev)
        dgamma, dbeta = torch.empty(D, dtype=f32, device=dev), torch.empty(D, dtype=f32, device=dev)
        lddx = D
    else:
        dX, dgamma, dbeta = out
        lddx = _matrix(dX, "dX", dev, dtype, M, D)
    L = lib()
    ws, wsp, wsb = _scratch(ws, L.qg_workspace_size(QG_OP_LAYER_NORM_BACKWARD, 1, 1, D), dev)
    _check("layer_norm_backward", L.layer_norm_backward(
        dt, M, D, dY.data_ptr(), lddy, X.data_ptr(), ldx, g, wd, _vector(mean, "mean", M, f32, dev),
        _vector(rstd, "rstd", M, f32, dev), dX.data_ptr(), lddx, _vector(dgamma, "dgamma", D, f32, dev),
        _vector(dbeta, "dbeta", D, f32, dev), wsp, wsb, _raw_stream(dev)))
    return dX, dgamma, dbeta
