"""Python binding of libw4 (argument marshalling only).

Every function here forwards torch tensors' device pointers, sizes and the
current CUDA stream to the C ABI declared in ``include/w4.h``; all arithmetic
runs in the library's CUDA kernels.  There is no fallback: if ``libw4.so`` is
not built, importing this module raises.

Names follow the C ABI: ``w4_quantize`` (and ``w4_quantize_symmetric``), ``w4_pack``, ``w4a16_gemm``,
``w4a16_gemm_workspace_size``, ``w4a16_gemm_host``, ``w4a16_gemm_decode_static``,
``w4a16_linear``, ``w4a16_gated``, ``w4a16_linear_grad``, ``w4a16_gated_grad``,
``w4_device_error``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libw4.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libw4.so is not built ({_LIB_PATH}); run weight_only_int4_w4_b200.build.build_library()")

_lib = ctypes.CDLL(_LIB_PATH)
_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_lib.w4_quantize.argtypes = [_P, ctypes.c_int, _P, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P]
_lib.w4_quantize_symmetric.argtypes = [_P, ctypes.c_int, _P, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P]
_lib.w4_pack.argtypes = [_P, _I64, _I64, _P, _P]
_lib.w4a16_gemm.argtypes = [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, ctypes.c_int,
                            _P, _SZ, _P]
_lib.w4a16_gemm_host.argtypes = [_P, _P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P,
                                 ctypes.c_int, _P, _SZ, _P]
_lib.w4a16_gemm_host_async.argtypes = _lib.w4a16_gemm_host.argtypes
_lib.w4a16_gemm_decode_static.argtypes = [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P,
                                          ctypes.c_int, _P]
_lib.w4a16_gemm_decode_static_capacity.argtypes = []
_lib.w4a16_gemm_decode_static_capacity.restype = _SZ
_lib.w4_awq_search.argtypes = [_P, _I64, _I64, ctypes.c_int, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P, _P, _P,
                               _P, _SZ, _P]
_lib.w4_awq_search_workspace_size.argtypes = [_I64, _I64, _I64, ctypes.c_int]
_lib.w4_awq_search_workspace_size.restype = _SZ
_lib.w4_quantize_outliers.argtypes = [_P, _P, _I64, _I64, ctypes.c_int, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P,
                                      _SZ, _P]
_lib.w4_outliers_workspace_size.argtypes = [_I64]
_lib.w4_outliers_workspace_size.restype = _SZ
_lib.w4_outliers_default_count.argtypes = [_I64, _I64]
_lib.w4_outliers_default_count.restype = _I64
_lib.w4a16_gemm_outliers.argtypes = [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P,
                                     _P, ctypes.c_int, _P, _SZ, _P]
_lib.w4_quantize_gptq.argtypes = [_P, _I64, _I64, ctypes.c_int, _P, ctypes.c_int, _I64, ctypes.c_double, _P, _P, _P,
                                  _P, _P, _SZ, _P]
_lib.w4_gptq_workspace_size.argtypes = [_I64, _I64]
_lib.w4_gptq_workspace_size.restype = _SZ
_lib.w4a16_gemm_workspace_size.argtypes = [_I64, _I64, _I64]
_lib.w4a16_gemm_workspace_size.restype = _SZ


_I = ctypes.c_int
_lib.w4a16_linear.argtypes = [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _SZ, _P]
_lib.w4a16_gated.argtypes = [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P, _SZ, _P]
_lib.w4a16_linear_grad.argtypes = [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _SZ, _P]
_lib.w4a16_gated_grad.argtypes = _lib.w4a16_linear_grad.argtypes
for _f in ("w4a16_linear", "w4a16_gated", "w4a16_linear_grad", "w4a16_gated_grad"):
    getattr(_lib, _f).restype = _I
    getattr(_lib, _f + "_workspace_size").argtypes = [_I64, _I64, _I64]
    getattr(_lib, _f + "_workspace_size").restype = _SZ


class GemmItem(ctypes.Structure):
    """w4_gemm_item of include/w4.h: one matmul of a host-buffer batch."""
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64), ("group", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("packed", _P), ("scales", _P), ("zeros", _P), ("awq_s", _P),
                ("x_offset", _SZ), ("y_offset", _SZ)]


_lib.w4a16_gemm_host_batch_async.argtypes = [ctypes.POINTER(GemmItem), ctypes.c_int, _P, _P, _SZ, _P, _P, _SZ, _P,
                                             _SZ, _P]
_lib.w4_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
_lib.w4_status_string.argtypes = [ctypes.c_int]
_lib.w4_status_string.restype = ctypes.c_char_p
_lib.w4_last_error.restype = ctypes.c_char_p
for _f in ("w4_quantize", "w4_quantize_symmetric", "w4_awq_search", "w4_quantize_outliers", "w4a16_gemm_outliers",
           "w4_quantize_gptq",
           "w4_pack", "w4a16_gemm", "w4a16_gemm_host", "w4a16_gemm_host_async", "w4a16_gemm_host_batch_async",
           "w4a16_gemm_decode_static", "w4_device_error"):
    getattr(_lib, _f).restype = ctypes.c_int

W4_OK, W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED, W4_ERR_CUDA = 0, 1, 2, 3
W4_F32, W4_F16, W4_BF16 = 0, 1, 2
_DT = {torch.float32: W4_F32, torch.float16: W4_F16, torch.bfloat16: W4_BF16}
GROUP = 128

LIB_PATH = _LIB_PATH
lib = _lib


class W4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.w4_last_error().decode()
        super().__init__(f"{where}: {_lib.w4_status_string(status).decode()}: {msg}")


def _check(status: int, where: str):
    if status != W4_OK:
        raise W4Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def w4_status_string(status: int) -> str:
    return _lib.w4_status_string(status).decode()


def w4_quantize(W: torch.Tensor, awq_s: torch.Tensor | None = None, group: int = GROUP,
                return_codes: bool = False, stream=None, symmetric: bool = False, out=None):
    """Quantize + pack W [N, K] (fp32/fp16/bf16, CUDA).  Returns (packed u8 [N,K/2],
    scales f16 [N,K/G], zeros f16 [N,K/G]) and, with return_codes, codes u8 [N,K].
    symmetric=True calls w4_quantize_symmetric (codes q + 8, q in [-7, 7]).
    out = (packed, scales, zeros) writes into caller-owned tensors of those shapes."""
    assert W.is_cuda and W.dim() == 2 and W.is_contiguous() and W.dtype in _DT
    N, K = W.shape
    dev = W.device
    if out is not None:
        packed, scales, zeros = out
        assert packed.shape == (N, K // 2) and scales.shape == (N, K // group) and zeros.shape == (N, K // group)
    else:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // group), dtype=torch.float16, device=dev)
        zeros = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev) if return_codes else None
    if awq_s is not None:
        assert awq_s.is_cuda and awq_s.dtype == torch.float32 and awq_s.is_contiguous()
    fn, name = (_lib.w4_quantize_symmetric, "w4_quantize_symmetric") if symmetric else (_lib.w4_quantize, "w4_quantize")
    _check(fn(_ptr(W), _DT[W.dtype], _ptr(awq_s), N, K, group, _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(codes),
              _stream(stream)), name)
    return (packed, scales, zeros, codes) if return_codes else (packed, scales, zeros)


def w4_pack(codes: torch.Tensor, stream=None) -> torch.Tensor:
    assert codes.is_cuda and codes.dtype == torch.uint8 and codes.dim() == 2 and codes.is_contiguous()
    N, K = codes.shape
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    _check(_lib.w4_pack(_ptr(codes), N, K, _ptr(packed), _stream(stream)), "w4_pack")
    return packed


def w4a16_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.w4a16_gemm_workspace_size(M, N, K))


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def workspace(M: int, N: int, K: int, device, stream=None) -> torch.Tensor | None:
    """A workspace (cached per device and stream) large enough for (M, N, K), zero-filled
    when allocated.  Every call leaves its counters zero again, so it can be reused.  Calls that
    are given it as `ws` must not overlap, not even on the host (a call may be several
    launches); calls without `ws` see to that themselves."""
    need = w4a16_gemm_workspace_size(M, N, K)
    if need == 0:
        return None
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (torch.device(device), s.cuda_stream)
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < need:
            with torch.cuda.stream(s):  # zeroed there before its first use, and given back there
                buf = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
    return buf


_stream_locks: dict = {}


def _stream_lock(dev: int, raw: int):
    """Held from taking a cached workspace until the call's last launch: a call is several launches
    that hand data on through it, and other threads run during the library's call.  Re-entrant,
    since a finalizer that runs while the workspace is allocated may make a call of its own."""
    return _stream_locks.get((dev, raw)) or _stream_locks.setdefault((dev, raw), threading.RLock())


def _own_workspace(call, M, N, K, device, stream):
    """call(ws) with the cached workspace, one call at a time on it."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    with _stream_lock(device.index, s.cuda_stream):
        return call(workspace(M, N, K, device, stream))


def w4a16_gemm(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
               awq_s: torch.Tensor | None = None, out_dtype=torch.float32, out: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, group: int = GROUP, stream=None) -> torch.Tensor:
    """Y = X . W^T with W^ dequantized on the fly.  X [M,K] fp16/bf16 (CUDA)."""
    assert X.is_cuda and X.dim() == 2 and X.is_contiguous() and X.dtype in (torch.float16, torch.bfloat16)
    M, K = X.shape
    N = packed.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=X.device)
    if ws is None and w4a16_gemm_workspace_size(M, N, K):
        return _own_workspace(lambda w: w4a16_gemm(X, packed, scales, zeros, awq_s, out=out, ws=w, group=group,
                                                   stream=stream), M, N, K, X.device, stream)
    _check(_lib.w4a16_gemm(_ptr(X), _DT[X.dtype], M, N, K, group, _ptr(packed), _ptr(scales), _ptr(zeros),
                           _ptr(awq_s), _ptr(out), _DT[out.dtype], _ptr(ws), 0 if ws is None else ws.numel(),
                           _stream(stream)), "w4a16_gemm")
    return out


def w4a16_gemm_host(X_host: torch.Tensor, X_dev: torch.Tensor, packed, scales, zeros, Y_host: torch.Tensor,
                    Y_dev: torch.Tensor, awq_s=None, ws=None, group: int = GROUP, stream=None,
                    wait: bool = True) -> torch.Tensor:
    """End-to-end call with pinned host X and Y: H2D copy, fused GEMM, D2H copy, and
    (wait=True) a wait for the stream.  With wait=False the work is only enqueued
    (w4a16_gemm_host_async): Y_host is valid after the caller synchronizes the stream."""
    M, K = X_host.shape
    N = packed.shape[0]
    if ws is None and w4a16_gemm_workspace_size(M, N, K):
        return _own_workspace(lambda w: w4a16_gemm_host(X_host, X_dev, packed, scales, zeros, Y_host, Y_dev, awq_s, w,
                                                        group, stream, wait), M, N, K, X_dev.device, stream)
    fn = _lib.w4a16_gemm_host if wait else _lib.w4a16_gemm_host_async
    _check(fn(_ptr(X_host), _ptr(X_dev), _DT[X_host.dtype], M, N, K, group, _ptr(packed), _ptr(scales), _ptr(zeros),
              _ptr(awq_s), _ptr(Y_host), _ptr(Y_dev), _DT[Y_host.dtype], _ptr(ws), 0 if ws is None else ws.numel(),
              _stream(stream)), "w4a16_gemm_host" if wait else "w4a16_gemm_host_async")
    return Y_host


def gemm_batch(items) -> ctypes.Array:
    """The w4_gemm_item array for w4a16_gemm_host_batch: one entry per matmul, each a dict
    with M, N, K, packed, scales, zeros, x_offset and y_offset (bytes into the staging
    buffers), and optionally awq_s, group (128), x_dtype (torch.bfloat16) and y_dtype
    (torch.float32).  Build it once and reuse it while the weights stay in place."""
    arr = (GemmItem * len(items))()
    for a, it in zip(arr, items):
        a.M, a.N, a.K = it["M"], it["N"], it["K"]
        a.group = it.get("group", GROUP)
        a.x_dtype = _DT[it.get("x_dtype", torch.bfloat16)]
        a.y_dtype = _DT[it.get("y_dtype", torch.float32)]
        a.packed, a.scales, a.zeros = it["packed"].data_ptr(), it["scales"].data_ptr(), it["zeros"].data_ptr()
        a.awq_s = it["awq_s"].data_ptr() if it.get("awq_s") is not None else None
        a.x_offset, a.y_offset = it["x_offset"], it["y_offset"]
    return arr


def w4a16_gemm_host_batch(batch: ctypes.Array, X_host: torch.Tensor, X_dev: torch.Tensor, Y_host: torch.Tensor,
                          Y_dev: torch.Tensor, ws=None, stream=None, wait: bool = True):
    """Independent matmuls with pinned host activations and outputs in one call
    (w4a16_gemm_host_batch_async): one copy of X_host into X_dev, the matmuls of `batch`
    (from gemm_batch) in order, one copy of Y_dev into Y_host.  The staging buffers are
    byte views (any dtype); with wait=False Y_host is valid after the caller
    synchronizes the stream."""
    xb, yb = X_host.numel() * X_host.element_size(), Y_host.numel() * Y_host.element_size()
    assert X_dev.numel() * X_dev.element_size() >= xb and Y_dev.numel() * Y_dev.element_size() >= yb
    _check(_lib.w4a16_gemm_host_batch_async(batch, len(batch), _ptr(X_host), _ptr(X_dev), xb, _ptr(Y_host),
                                            _ptr(Y_dev), yb, _ptr(ws), 0 if ws is None else ws.numel(),
                                            _stream(stream)), "w4a16_gemm_host_batch_async")
    if wait:
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return Y_host


def w4a16_gemm_decode_static(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                             awq_s: torch.Tensor | None = None, out_dtype=torch.float32,
                             out: torch.Tensor | None = None, group: int = GROUP, stream=None) -> torch.Tensor:
    """Decode-shape Y = X . W^T using the library's own fixed scratch (no workspace
    argument).  Calls on one device must not overlap in time."""
    assert X.is_cuda and X.dim() == 2 and X.is_contiguous() and X.dtype in (torch.float16, torch.bfloat16)
    M, K = X.shape
    N = packed.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=X.device)
    _check(_lib.w4a16_gemm_decode_static(_ptr(X), _DT[X.dtype], M, N, K, group, _ptr(packed), _ptr(scales),
                                         _ptr(zeros), _ptr(awq_s), _ptr(out), _DT[out.dtype], _stream(stream)),
           "w4a16_gemm_decode_static")
    return out


def w4a16_gemm_decode_static_capacity() -> int:
    return int(_lib.w4a16_gemm_decode_static_capacity())


def w4_quantize_outliers(W: torch.Tensor, count: int | None = None, awq_s: torch.Tensor | None = None,
                         group: int = GROUP, stream=None):
    """Dense + sparse split of W [N,K] fp32 (CUDA): the `count` largest |w| in fp16 CSR (None: the
    library's default, w4_outliers_default_count), the rest quantized.
    Returns (packed, scales, zeros, (row_ptr, col, val))."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous()
    N, K = W.shape
    dev = W.device
    cap = int(_lib.w4_outliers_default_count(N, K)) if count is None else int(count)
    count = 0 if count is None else int(count)
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    zeros = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    ws = torch.zeros(int(_lib.w4_outliers_workspace_size(N)), dtype=torch.uint8, device=dev)
    cap += 1024
    while True:
        col = torch.empty(cap, dtype=torch.int32, device=dev)
        val = torch.empty(cap, dtype=torch.float16, device=dev)
        nnz = ctypes.c_int64(0)
        st = _lib.w4_quantize_outliers(_ptr(W), _ptr(awq_s), N, K, group, count, _ptr(packed), _ptr(scales),
                                       _ptr(zeros), _ptr(row_ptr), _ptr(col), _ptr(val), cap,
                                       ctypes.cast(ctypes.pointer(nnz), _P), _ptr(ws), ws.numel(), _stream(stream))
        if st == W4_ERR_INVALID_ARG and nnz.value > cap:
            cap = nnz.value
            continue
        _check(st, "w4_quantize_outliers")
        break
    return packed, scales, zeros, (row_ptr, col[: nnz.value], val[: nnz.value])


def w4a16_gemm_outliers(X: torch.Tensor, packed, scales, zeros, csr, awq_s=None, out_dtype=torch.float32,
                        out: torch.Tensor | None = None, ws: torch.Tensor | None = None, group: int = GROUP,
                        stream=None) -> torch.Tensor:
    """Y = X . (dequant(dense) + sparse)^T with the CSR from w4_quantize_outliers."""
    assert X.is_cuda and X.dim() == 2 and X.is_contiguous() and X.dtype in (torch.float16, torch.bfloat16)
    M, K = X.shape
    N = packed.shape[0]
    row_ptr, col, val = csr
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=X.device)
    if ws is None and w4a16_gemm_workspace_size(M, N, K):
        return _own_workspace(lambda w: w4a16_gemm_outliers(X, packed, scales, zeros, csr, awq_s, out=out, ws=w, group=group,
                                                            stream=stream), M, N, K, X.device, stream)
    _check(_lib.w4a16_gemm_outliers(_ptr(X), _DT[X.dtype], M, N, K, group, _ptr(packed), _ptr(scales), _ptr(zeros),
                                    _ptr(awq_s), _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(out), _DT[out.dtype],
                                    _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "w4a16_gemm_outliers")
    return out


def w4_quantize_gptq(W: torch.Tensor, Xcal: torch.Tensor, group: int = GROUP, damp_frac: float = 0.01,
                     return_codes: bool = False, stream=None):
    """GPTQ column sweep of W [N,K] fp32 with calibration Xcal [Mc,K] f16/bf16 (CUDA).
    Returns (packed, scales, zeros) and, with return_codes, codes u8 [N,K]."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous()
    assert Xcal.is_cuda and Xcal.dtype in (torch.float16, torch.bfloat16) and Xcal.is_contiguous()
    N, K = W.shape
    dev = W.device
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    zeros = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev) if return_codes else None
    ws = torch.empty(int(_lib.w4_gptq_workspace_size(N, K)), dtype=torch.uint8, device=dev)
    _check(_lib.w4_quantize_gptq(_ptr(W), N, K, group, _ptr(Xcal), _DT[Xcal.dtype], Xcal.shape[0], float(damp_frac),
                                 _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(codes), _ptr(ws), ws.numel(),
                                 _stream(stream)), "w4_quantize_gptq")
    return (packed, scales, zeros, codes) if return_codes else (packed, scales, zeros)


AWQ_EXPONENTS = tuple(round(-1.0 + 0.1 * i, 1) for i in range(21))  # -1.0, -0.9, ..., 1.0


def w4_awq_search(W: torch.Tensor, Xcal: torch.Tensor, alphas=AWQ_EXPONENTS, group: int = GROUP, stream=None):
    """AWQ exponent search on calibration activations.  W [N,K] fp32, Xcal [Mc,K] f16/bf16 (CUDA).
    Returns (awq_s fp32 [K] on the device, best exponent, errors list)."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous()
    assert Xcal.is_cuda and Xcal.dtype in (torch.float16, torch.bfloat16) and Xcal.is_contiguous()
    N, K = W.shape
    Mc = Xcal.shape[0]
    a = (ctypes.c_float * len(alphas))(*alphas)
    errs = (ctypes.c_double * len(alphas))()
    best = ctypes.c_int(-1)
    s = torch.empty(K, dtype=torch.float32, device=W.device)
    ws = torch.zeros(int(_lib.w4_awq_search_workspace_size(Mc, N, K, group)), dtype=torch.uint8, device=W.device)
    _check(_lib.w4_awq_search(_ptr(W), N, K, group, _ptr(Xcal), _DT[Xcal.dtype], Mc, ctypes.cast(a, _P), len(alphas),
                              _ptr(s), ctypes.cast(errs, _P), ctypes.cast(ctypes.pointer(best), _P), _ptr(ws),
                              ws.numel(), _stream(stream)), "w4_awq_search")
    return s, alphas[best.value], list(errs)


# ---------------------------------------------------------------- fused operators
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}  # w4_act of include/w4.h


def w4a16_linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.w4a16_linear_workspace_size(M, N, K))


def w4a16_gated_workspace_size(M: int, F: int, K: int) -> int:
    return int(_lib.w4a16_gated_workspace_size(M, F, K))


def w4a16_linear_grad_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.w4a16_linear_grad_workspace_size(M, N, K))


def w4a16_gated_grad_workspace_size(M: int, F: int, K: int) -> int:
    return int(_lib.w4a16_gated_grad_workspace_size(M, F, K))


_fused_ws: dict = {}
_raw_stream = torch._C._cuda_getCurrentRawStream
_DECODE_TOKENS = 8  # up to here, with groups of 128, a forward call needs no workspace
_X_DT = {torch.float16: W4_F16, torch.bfloat16: W4_BF16}


def _fused_workspace(need: int, dev, raw: int, stream):
    """Scratch of a fused call: cached per device and stream, like workspace(); while the stream
    is being captured into a graph, a buffer of the graph's own, so that no two graphs and
    no later call share one."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _fused_workspace(need, dev, raw, None)
    capturing = torch.cuda.is_current_stream_capturing()
    buf = None if capturing else _fused_ws.get((dev, raw))
    if buf is None or buf.numel() < need:
        buf = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=dev)
        if not capturing:
            _fused_ws[(dev, raw)] = buf
    return buf


def _bad(name, what):
    raise ValueError(f"{name}: {what}")


def _fused_layer(name, X, packed, scales, zeros, awq_s, group, stream):
    """The checks that every fused call shares; returns (device index, M, N, K)."""
    dev = X.get_device()
    if dev < 0 or X.dim() != 2 or X.dtype not in _X_DT or not X.is_contiguous():
        _bad(name, "the activations or gradients are a contiguous 2-D CUDA tensor in fp16 or bf16")
    if packed.dtype is not torch.uint8 or packed.dim() != 2 or not packed.is_contiguous() or packed.get_device() != dev:
        _bad(name, "packed is a contiguous uint8 [N, K/2] tensor on the activations' device")
    if type(group) is not int or group < 1:
        _bad(name, "group is a positive number")
    N, K = packed.shape
    K *= 2
    shape = (N, K // group)
    for t in (scales, zeros):
        if t.dtype is not torch.float16 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
            _bad(name, f"scales and zeros are contiguous fp16 tensors of shape {shape} on the activations' device")
    if awq_s is not None:
        _vector(name, "awq_s", awq_s, K, dev)
    if stream is not None and stream.device_index != dev:
        _bad(name, "stream is one of the activations' device")
    return dev, X.shape[0], N, K


def _vector(name, what, t, n, dev):
    if t.dtype is not torch.float32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        _bad(name, f"{what} is a contiguous fp32 tensor of {n} elements on the activations' device")


def _matrix(name, what, t, M, N, dtype, dev):
    if t.dtype is not dtype or t.shape != (M, N) or not t.is_contiguous() or t.get_device() != dev:
        _bad(name, f"{what} is a contiguous {dtype} tensor of shape [{M}, {N}] on the activations' device")


def _new(like, shape, dtype, stream):
    """A result tensor that belongs to the stream that writes it: one of the current stream's might
    lie where kernels still queued there read or write."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _output(name, out, M, N, out_dtype, like, dev, stream):
    if out is None:
        if out_dtype is not None and out_dtype not in _DT:
            _bad(name, "the output is fp32, fp16 or bf16")
        return _new(like, (M, N), out_dtype, stream)
    if out.dtype not in _DT or out_dtype not in (None, out.dtype):
        _bad(name, "out is fp32, fp16 or bf16, and of out_dtype if that is given")
    _matrix(name, "out", out, M, N, out.dtype, dev)
    return out


def _act(name, act):
    a = ACTS.get(act)
    return a if a is not None else _bad(name, f"act is one of {sorted(ACTS)}")


def _fused_call(name, fn, size_fn, sizes, dev, ws, stream, args):
    """Makes the C call on device `dev`: args and then the workspace and stream."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _fused_call(name, fn, size_fn, sizes, dev, ws, stream, args)
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    if ws is None:
        need = size_fn(*sizes) if size_fn is not None else 0
        if need:
            with _stream_lock(dev, raw):
                ws = _fused_workspace(need, dev, raw, stream)
                st = fn(*args, ws.data_ptr(), ws.numel(), raw)
            if st:
                raise W4Error(st, name)
            return
    elif ws.dtype is not torch.uint8 or not ws.is_contiguous() or ws.get_device() != dev:
        _bad(name, "ws is a contiguous uint8 tensor on the activations' device")
    st = fn(*args, 0, 0, raw) if ws is None else fn(*args, ws.data_ptr(), ws.numel(), raw)
    if st:
        raise W4Error(st, name)


def w4a16_linear(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                 awq_s: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "none",
                 residual: torch.Tensor | None = None, out_dtype=None, out: torch.Tensor | None = None,
                 save_preact: bool = False, group: int = GROUP, ws: torch.Tensor | None = None, stream=None):
    """Y = act(X . W^T + bias) + residual.  X [M,K] fp16/bf16 (CUDA), bias fp32 [N], residual [M,N] of
    the output's type (`out` may be the residual itself, but not X); Y in out_dtype (X's type by default).
    With save_preact, returns (Y, Z), Z = X . W^T + bias in X's type, for w4a16_linear_grad.
    With `stream`, the call runs there and the results belong to it, as if it were current.
    Without `ws`, the workspace is the binding's own, one per device and stream, and threads may share a
    stream.  Calls that share a given `ws` must not overlap in time: not on the device, and not on the
    host either (a call is several launches).
    Tensors that do not fit raise ValueError, what the library refuses raises W4Error."""
    name = "w4a16_linear"
    dev, M, N, K = _fused_layer(name, X, packed, scales, zeros, awq_s, group, stream)
    if X.shape[1] != K:
        _bad(name, f"X has {X.shape[1]} channels, the weights {K}")
    a = _act(name, act)
    if bias is not None:
        _vector(name, "bias", bias, N, dev)
    Y = _output(name, out, M, N, out_dtype, X, dev, stream)
    if residual is not None:
        _matrix(name, "residual", residual, M, N, Y.dtype, dev)
    Z = _new(X, (M, N), None, stream) if save_preact else None
    decode = M <= _DECODE_TOKENS and group == GROUP
    _fused_call(name, _lib.w4a16_linear, None if decode else _lib.w4a16_linear_workspace_size, (M, N, K), dev, ws, stream,
                (X.data_ptr(), _X_DT[X.dtype], M, N, K, group, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                 0 if awq_s is None else awq_s.data_ptr(), 0 if bias is None else bias.data_ptr(), a,
                 0 if residual is None else residual.data_ptr(), 0 if Z is None else Z.data_ptr(), Y.data_ptr(),
                 _DT[Y.dtype]))
    return (Y, Z) if save_preact else Y


def w4a16_gated(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                awq_s: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "silu", out_dtype=None,
                out: torch.Tensor | None = None, save_preact: bool = False, group: int = GROUP,
                ws: torch.Tensor | None = None, stream=None):
    """H = act(G) * U with [G U] = X . W^T + bias; the weights' rows are F gate rows, then F up rows.
    H [M,F] in out_dtype (X's type by default).  With save_preact, returns (H, Z), Z = [G U]
    [M,2F] in X's type, for w4a16_gated_grad.  Errors as w4a16_linear."""
    name = "w4a16_gated"
    dev, M, N, K = _fused_layer(name, X, packed, scales, zeros, awq_s, group, stream)
    if X.shape[1] != K:
        _bad(name, f"X has {X.shape[1]} channels, the weights {K}")
    if N % 2:
        _bad(name, "the weights have an even number of rows, gate rows first")
    a = _act(name, act)
    if bias is not None:
        _vector(name, "bias", bias, N, dev)
    F = N // 2
    H = _output(name, out, M, F, out_dtype, X, dev, stream)
    Z = _new(X, (M, N), None, stream) if save_preact else None
    decode = M <= _DECODE_TOKENS and group == GROUP
    _fused_call(name, _lib.w4a16_gated, None if decode else _lib.w4a16_gated_workspace_size, (M, F, K), dev, ws, stream,
                (X.data_ptr(), _X_DT[X.dtype], M, F, K, group, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                 0 if awq_s is None else awq_s.data_ptr(), 0 if bias is None else bias.data_ptr(), a,
                 0 if Z is None else Z.data_ptr(), H.data_ptr(), _DT[H.dtype]))
    return (H, Z) if save_preact else H


def w4a16_linear_grad(dY: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      awq_s: torch.Tensor | None = None, preact: torch.Tensor | None = None, act: str = "none",
                      dbias: bool = False, out_dtype=None, out: torch.Tensor | None = None, group: int = GROUP,
                      ws: torch.Tensor | None = None, stream=None):
    """dX [M,K] = (dY * act'(Z)) . W^ for frozen weights.  dY [M,N] fp16/bf16 (CUDA), preact = Z [M,N] of
    its type (not needed for act "none").  With dbias, returns (dX, dbias fp32 [N]).  Errors as
    w4a16_linear."""
    return _grad("w4a16_linear_grad", False, _lib.w4a16_linear_grad, _lib.w4a16_linear_grad_workspace_size, dY, packed,
                 scales, zeros, awq_s, preact, act, dbias, out_dtype, out, group, ws, stream)


def w4a16_gated_grad(dH: torch.Tensor, preact: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                     zeros: torch.Tensor, awq_s: torch.Tensor | None = None, act: str = "silu", dbias: bool = False,
                     out_dtype=None, out: torch.Tensor | None = None, group: int = GROUP,
                     ws: torch.Tensor | None = None, stream=None):
    """dX [M,K] = [dG dU] . W^ with dG = dH * U * act'(G), dU = dH * act(G), from preact = [G U] [M,2F] of
    dH's type.  With dbias, returns (dX, dbias fp32 [2F]).  Errors as w4a16_linear."""
    return _grad("w4a16_gated_grad", True, _lib.w4a16_gated_grad, _lib.w4a16_gated_grad_workspace_size, dH, packed,
                 scales, zeros, awq_s, preact, act, dbias, out_dtype, out, group, ws, stream)


def _grad(name, gated, fn, size_fn, dY, packed, scales, zeros, awq_s, preact, act, dbias, out_dtype, out, group, ws,
          stream):
    dev, M, N, K = _fused_layer(name, dY, packed, scales, zeros, awq_s, group, stream)
    if gated and N % 2:
        _bad(name, "the weights have an even number of rows, gate rows first")
    width = N // 2 if gated else N
    if dY.shape[1] != width:
        _bad(name, f"the gradient has {dY.shape[1]} channels, the weights give {width}")
    a = _act(name, act)
    if preact is not None:
        _matrix(name, "preact", preact, M, N, dY.dtype, dev)
    dX = _output(name, out, M, K, out_dtype, dY, dev, stream)
    db = _new(dY, (N,), torch.float32, stream) if dbias else None
    _fused_call(name, fn, size_fn, (M, width, K), dev, ws, stream,
                (dY.data_ptr(), _X_DT[dY.dtype], M, width, K, group, packed.data_ptr(), scales.data_ptr(),
                 zeros.data_ptr(), 0 if awq_s is None else awq_s.data_ptr(), 0 if preact is None else preact.data_ptr(),
                 a, dX.data_ptr(), _DT[dX.dtype], 0 if db is None else db.data_ptr()))
    return (dX, db) if dbias else dX


def w4_device_error() -> int:
    flag = ctypes.c_int(0)
    _check(_lib.w4_device_error(ctypes.byref(flag)), "w4_device_error")
    return flag.value
