"""Python binding of libtq.so: the C entry points under the same names.

Argument marshalling only.  Host functions take numpy arrays; device functions
take torch tensors that already live on the GPU and pass their data pointers
and the current HIP stream.  Every status other than TQ_OK raises ``TQError``.
Importing this module raises ``ImportError`` when libtq.so has not been built:
there is no fallback.
"""

from __future__ import annotations

import ctypes as C
import functools
import math
import os
import types
import warnings

import numpy as np

# One HIP runtime per process.  libtq.so needs libamdhip64.so.7, and the torch
# wheel carries its own copy of that library (and of the HSA runtime).  If
# libtq.so were loaded first, the system copy would be mapped and torch would
# then map its own: two runtimes claiming one GPU, which crashes on the first
# device allocation.  Importing torch first lets the loader resolve libtq.so's
# dependency to the copy torch already mapped.
try:
    import torch as _torch  # noqa: F401
except ImportError:  # host-only use without torch: the system runtime is the only one
    _torch = None

# TQ_LIBRARY names another build of the same library (the sanitizer variant
# of build_lib); by default the in-tree libtq.so next to this file.
_LIB_PATH = os.environ.get("TQ_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libtq.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing; build it with "
                      "`python -m bit_mixed_precision_amd.build_lib`")
lib = C.CDLL(_LIB_PATH)

TQ_OK, TQ_ERR_NULL, TQ_ERR_SHAPE, TQ_ERR_VALUE, TQ_ERR_ALIGN, TQ_ERR_DEVICE, TQ_ERR_UNSUPPORTED = \
    0, -1, -2, -3, -4, -5, -6
TQ_SRC_TERNARY_I8, TQ_SRC_LATENT_F32 = 0, 1
TQ_PATH_AUTO, TQ_PATH_SKINNY, TQ_PATH_TILED, TQ_PATH_SIMPLE = 0, 1, 2, 3
TQ_F16, TQ_BF16, TQ_F32 = 0, 1, 2
TQ_ROPE_NONE, TQ_ROPE_LINEAR, TQ_ROPE_BASE, TQ_ROPE_PARTS = 0, 1, 2, 3

_P, _I64, _I, _D = C.c_void_p, C.c_int64, C.c_int, C.c_double

#: Every symbol include/tq.h declares, with (restype, argtypes).
SIGNATURES = {
    "tq_status_string": (C.c_char_p, [_I]),
    "tq_abi_version": (_I, []),
    "tq_tq2_bytes": (_I64, [_I64, _I64]),
    "tq_tq1_ldq": (_I64, [_I64]),
    "tq_num_scales": (_I64, [_I64, _I64]),
    "tq_ternarize_f32": (_I, [_P, _I64, _I64, _D, _P, _P]),
    "tq_pack_tq2": (_I, [_I, _P, _I64, _I64, _D, _P, _P, _P]),
    "tq_pack_tq1": (_I, [_I, _P, _I64, _I64, _D, _I64, _P, _P, _P]),
    "tq_unpack_tq2": (_I, [_P, _I64, _I64, _P]),
    "tq_unpack_tq1": (_I, [_P, _I64, _I64, _I64, _P]),
    "tq_gemm_tq2": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "tq_gemm_tq1": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P]),
    "tq_kernel_name": (_I, [_I, _I64, _I64, _I64, _I, C.c_char_p, _I64]),
    "tq_gemm_tq2_ex": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "tq_gemm_tq1_ex": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I, _P]),
    "tq_gemm_tq2_tiled": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P]),
    "tq_gemm_tq2_tile": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _I, _P]),
    "tq_gemm_tq2_wide": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _I, _P]),
    "tq_gemm_tq2_swiglu": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "tq_gemm_tq2_bwd_x": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "tq_stream_read": (_I, [_P, _I64, _P, _P]),
    "tq_ste_grad_w": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "tq_transcode_tq1_tq2": (_I, [_P, _I64, _I64, _I64, _P, _P]),
    "tq_tq1_transcode_min_m": (_I64, [_I64, _I64]),
    "tq_gemm_tq1_ws": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "tq_gemm_tq1_tile": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I, _I, _I, _I, _P]),
    "tq_pack_dev_workspace_bytes": (_I64, [_I64, _I64]),
    "tq_pack_tq2_dev": (_I, [_P, _I64, _I64, C.c_double, _P, _P, _P, _P, _P, _I64, _P]),
    "tq_pack_tq1_dev": (_I, [_P, _I64, _I64, C.c_double, _I64, _P, _P, _P, _P, _P, _I64, _P]),
    "tq_pack_tq2_dev_noalloc": (_I, [_P, _I64, _I64, C.c_double, _P, _P, _P, _P, _P]),
    "tq_rope_table": (_I, [_I64, _I64, _D, _I, _D, _D, _D, _D, _D, _P]),
    "tq_rope": (_I, [_I, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64,
                     _I, _I, _P]),
    "tq_rope_append": (_I, [_I, _P, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _P, _I64,
                            _I64, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I, _P]),
    "tq_paged_attention": (_I, [_I, _P, _I64, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _P,
                                _I64, _P, _I64, _I64, _I64, _I64, _D, _I64, _P, _P, _P, _I64,
                                _P]),
    "tq_paged_attention_workspace": (_I64, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "tq_pages_fork": (_I, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _P,
                           _P, _P, _I64, _P]),
    "tq_pages_grow": (_I, [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P]),
    "tq_pages_compact": (_I, [_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64,
                              _P]),
    "tq_pages_copy": (_I, [_P, _I64, _I64, _I64, _P, _P, _I64, _P]),
    "tq_pages_workspace": (_I64, [_I64, _I64]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


# The decode-side calls in their common form, compiled (csrc_decode/tq_torch.cc);
# each returns None for what it leaves to the functions below.  Those serve every
# call, on the same kernels: without the compiled forms, or where they were built for
# another torch, a call takes some 5 us more of the host, and nothing else changes.
def _compiled_calls():
    try:
        from . import _tq_torch as fast
        built_for = getattr(fast, "torch_version", None)
        if built_for != _torch.__version__:
            raise ImportError(f"built for torch {built_for}, this is {_torch.__version__}")
    except ImportError as e:
        warnings.warn(f"_tq_torch.so is missing or does not load ({e}): the decode-side calls are "
                      "made from Python; build it with "
                      "`python -m bit_mixed_precision_amd.build_lib`", RuntimeWarning, stacklevel=3)
        return types.SimpleNamespace(**{n: lambda *a: None for n in (
            "rope", "rope_append", "paged_attention", "pages_fork", "pages_grow",
            "pages_compact")})
    fast.bind(getattr(_torch._C, "_cuda_getCurrentRawStream", lambda index: 0),
              {n: C.cast(getattr(lib, n), C.c_void_p).value for n in SIGNATURES})
    return fast


if _torch is not None:
    _fast = _compiled_calls()


class TQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {tq_status_string(status)} ({status})")


def _check(status: int, where: str) -> None:
    if status != TQ_OK:
        raise TQError(status, where)


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()  # torch tensor


def tq_status_string(status: int) -> str:
    return lib.tq_status_string(status).decode()


def tq_abi_version() -> int:
    return lib.tq_abi_version()


def tq_tq2_bytes(N: int, K: int) -> int:
    return lib.tq_tq2_bytes(N, K)


def tq_tq1_ldq(K: int) -> int:
    return lib.tq_tq1_ldq(K)


def tq_num_scales(N: int, K: int) -> int:
    return lib.tq_num_scales(N, K)


# ------------------------------------------------------------------ host

def tq_ternarize_f32(W: np.ndarray, eps: float = 1e-5):
    """(T int8 [N][K], gamma) for float32 latents W [N][K]."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    T = np.empty((N, K), dtype=np.int8)
    g = C.c_double(0.0)
    _check(lib.tq_ternarize_f32(_ptr(W), N, K, float(eps), _ptr(T), C.byref(g)), "tq_ternarize_f32")
    return T, g.value


def _src(W):
    W = np.asarray(W)
    if W.dtype == np.int8:
        return TQ_SRC_TERNARY_I8, np.ascontiguousarray(W)
    if W.dtype == np.float32:
        return TQ_SRC_LATENT_F32, np.ascontiguousarray(W)
    raise TypeError("W must be int8 trits or float32 latents")


def tq_pack_tq2(W: np.ndarray, eps: float = 1e-5):
    """Pack int8 trits or float32 latents W [N][K].

    Returns (qs uint8 [N][K/4], scales fp16 [N][K/256] or None, gamma or None);
    scales and gamma come back only for latents (fp16(gamma) in every block).
    """
    kind, W = _src(W)
    N, K = W.shape
    qs = np.empty((N, max(K // 4, 0)), dtype=np.uint8)
    scales = np.empty((N, max(K // 256, 0)), dtype=np.float16) if kind == TQ_SRC_LATENT_F32 else None
    g = C.c_double(0.0)
    _check(lib.tq_pack_tq2(kind, _ptr(W), N, K, float(eps), _ptr(qs), _ptr(scales), C.byref(g)),
           "tq_pack_tq2")
    return qs, scales, (g.value if scales is not None else None)


def tq_pack_tq1(W: np.ndarray, eps: float = 1e-5, ldq: int | None = None):
    """Like tq_pack_tq2 with the 1.6-bit packing; qs is uint8 [N][ldq]."""
    kind, W = _src(W)
    N, K = W.shape
    if ldq is None:
        ldq = tq_tq1_ldq(K)
    qs = np.empty((N, max(ldq, 0)), dtype=np.uint8)
    scales = np.empty((N, max(K // 256, 0)), dtype=np.float16) if kind == TQ_SRC_LATENT_F32 else None
    g = C.c_double(0.0)
    _check(lib.tq_pack_tq1(kind, _ptr(W), N, K, float(eps), ldq, _ptr(qs), _ptr(scales),
                           C.byref(g)), "tq_pack_tq1")
    return qs, scales, (g.value if scales is not None else None)


def tq_unpack_tq2(qs: np.ndarray, K: int) -> np.ndarray:
    qs = np.ascontiguousarray(qs, dtype=np.uint8)
    N = qs.shape[0]
    if qs.shape[1] * 4 != K:
        raise ValueError("qs does not hold K/4 bytes per row")
    T = np.empty((N, K), dtype=np.int8)
    _check(lib.tq_unpack_tq2(_ptr(qs), N, K, _ptr(T)), "tq_unpack_tq2")
    return T


def tq_unpack_tq1(qs: np.ndarray, K: int) -> np.ndarray:
    qs = np.ascontiguousarray(qs, dtype=np.uint8)
    N, ldq = qs.shape
    T = np.empty((N, K), dtype=np.int8)
    _check(lib.tq_unpack_tq1(_ptr(qs), N, K, ldq, _ptr(T)), "tq_unpack_tq1")
    return T


# ------------------------------------------------------------------ device

_DTYPES = {"f16": "float16", "bf16": "bfloat16", "f32": "float32", "u8": "uint8",
           "i32": "int32"}


_DT = {k: getattr(_torch, v) for k, v in _DTYPES.items()} if _torch is not None else {}


def _need(t, name, dtype, shape=None, where=""):
    """Check one device-tensor argument before its pointer reaches the C ABI,
    which receives bare pointers and cannot check sizes itself: a buffer that
    is too small would be read or written past its end.  Order: type and dtype
    (TQ_ERR_VALUE), rank, shape and contiguity (TQ_ERR_SHAPE), then device
    (TQ_ERR_DEVICE), so that every check but the last also runs without a GPU."""
    import torch
    if not torch.is_tensor(t):
        raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be a torch tensor")
    if t.dtype != _DT[dtype]:
        raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be {_DTYPES[dtype]}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} has shape {tuple(t.shape)}, "
                                    f"expected {tuple(shape)}")
    if not t.is_contiguous():
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be contiguous (row-major)")
    return t


def _on_gpu(where, *named):
    """Every (name, tensor) on a GPU, all on the first one's device; run after
    the dtype and shape checks of every argument."""
    first = named[0][1]
    for name, t in named:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise TQError(TQ_ERR_DEVICE, f"{where}: {name} is on {t.device}, not on a GPU")
        if t.device != first.device:
            raise TQError(TQ_ERR_DEVICE, f"{where}: {name} is on {t.device}, "
                                         f"{named[0][0]} on {first.device}")


def _rank2(t, name, where):
    import torch
    if not torch.is_tensor(t) or t.dim() != 2:
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be a 2-D tensor")
    return t.shape


def _stream(stream, device=None):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _out(Y, M, N, where, operands, name="Y"):
    """The output: Y checked as fp16 [M][N] when given, then every operand's
    device (``operands`` as (name, tensor) pairs); a new tensor on the first
    operand's device when Y is None (allocated only after every check)."""
    import torch
    if Y is not None:
        _need(Y, name, "f16", (M, N), where)
    _on_gpu(where, *operands, (name, Y))
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=operands[0][1].device)
    return Y


def _device_of(t):
    """Context that makes t's GPU the current HIP device for the C call."""
    import torch
    return torch.cuda.device(t.device)


def _gemm_operands(X, qs, scales, where, ldq_from_qs=False):
    """(M, N, K, ldq) of a product after checking X [M][K] fp16, qs [N][K/4]
    (TQ2) or [N][ldq] (TQ1) uint8 and scales [N][K/256] fp16."""
    M, K = _rank2(X, "X", where)
    N, qcols = _rank2(qs, "qs", where)
    _need(X, "X", "f16", None, where)
    _need(qs, "qs", "u8", (N, qcols if ldq_from_qs else K // 4), where)
    if not ldq_from_qs and qcols * 4 != K:
        raise TQError(TQ_ERR_SHAPE, f"{where}: qs has {qcols} bytes per row, expected K/4 = {K // 4}")
    _need(scales, "scales", "f16", (N, K // 256), where)
    return M, N, K, qcols


def tq_gemm_tq2_ex(X, qs, scales, path: int, Y=None, stream=None):
    """Y[M][N] = X[M][K] (s . T)^T for TQ2 weights qs [N][K/4]; tensors on the GPU."""
    where = "tq_gemm_tq2"
    M, N, K, _ = _gemm_operands(X, qs, scales, where)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq2_ex(_ptr(X), _ptr(qs), _ptr(scales), _ptr(Y), M, N, K, path,
                                  _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq1_ex(X, qs, scales, path: int, Y=None, stream=None):
    """Same as tq_gemm_tq2_ex for TQ1 weights qs [N][ldq] (ldq = qs.shape[1])."""
    where = "tq_gemm_tq1"
    M, N, K, ldq = _gemm_operands(X, qs, scales, where, ldq_from_qs=True)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq1_ex(_ptr(X), _ptr(qs), ldq, _ptr(scales), _ptr(Y), M, N, K, path,
                                  _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq2_tiled(X, qs, scales, mt: int, ng: int, kg: int, Y=None, stream=None):
    """tq_gemm_tq2 on the tiled kernel with an explicit (mt, ng, kg) tile."""
    where = "tq_gemm_tq2_tiled"
    M, N, K, _ = _gemm_operands(X, qs, scales, where)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq2_tiled(_ptr(X), _ptr(qs), _ptr(scales), _ptr(Y), M, N, K, mt, ng,
                                     kg, _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq2_swiglu(X, qs_gate, scales_gate, qs_up, scales_up, Y=None, stream=None):
    """silu(X G^T) * (X U^T) for TQ2 gate / up matrices, M <= 16, one launch."""
    where = "tq_gemm_tq2_swiglu"
    M, N, K, _ = _gemm_operands(X, qs_gate, scales_gate, where)
    _need(qs_up, "qs_up", "u8", tuple(qs_gate.shape), where)
    _need(scales_up, "scales_up", "f16", tuple(scales_gate.shape), where)
    Y = _out(Y, M, N, where, (("X", X), ("qs_gate", qs_gate), ("scales_gate", scales_gate),
                              ("qs_up", qs_up), ("scales_up", scales_up)))
    with _device_of(X):
        _check(lib.tq_gemm_tq2_swiglu(_ptr(X), _ptr(qs_gate), _ptr(scales_gate), _ptr(qs_up),
                                      _ptr(scales_up), _ptr(Y), M, N, K,
                                      _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq2_bwd_x(dY, qs, scales, dX=None, stream=None):
    """dX = dY (s . T): the input gradient of tq_gemm_tq2 (N % 8 == 0)."""
    where = "tq_gemm_tq2_bwd_x"
    M, N = _rank2(dY, "dY", where)
    _, qcols = _rank2(qs, "qs", where)
    K = qcols * 4
    _need(dY, "dY", "f16", None, where)
    _need(qs, "qs", "u8", (N, qcols), where)
    _need(scales, "scales", "f16", (N, K // 256), where)
    dX = _out(dX, M, K, where, (("dY", dY), ("qs", qs), ("scales", scales)), name="dX")
    with _device_of(dY):
        _check(lib.tq_gemm_tq2_bwd_x(_ptr(dY), _ptr(qs), _ptr(scales), _ptr(dX), M, N, K,
                                     _stream(stream, dY.device)), where)
    return dX


def tq_ste_grad_w(dY, X, dW=None, accumulate: bool = False, stream=None):
    """Latent-weight gradient under the straight-through estimator: dW [N][K]
    (float32) = dY^T X, or dW + dY^T X with accumulate (dW then required);
    dY fp16 [M][N], X fp16 [M][K]."""
    import torch
    where = "tq_ste_grad_w"
    M, N = _rank2(dY, "dY", where)
    M2, K = _rank2(X, "X", where)
    if M2 != M:
        raise TQError(TQ_ERR_SHAPE, f"{where}: dY has {M} rows, X {M2}")
    _need(dY, "dY", "f16", None, where)
    _need(X, "X", "f16", None, where)
    if dW is not None:
        _need(dW, "dW", "f32", (N, K), where)
    elif accumulate:
        raise TQError(TQ_ERR_NULL, f"{where}: accumulate needs dW")
    _on_gpu(where, ("dY", dY), ("X", X), ("dW", dW))
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=dY.device)
    with _device_of(dY):
        _check(lib.tq_ste_grad_w(_ptr(dY), _ptr(X), _ptr(dW), M, N, K, int(bool(accumulate)),
                                 _stream(stream, dY.device)), where)
    return dW


def tq_tq1_transcode_min_m(N: int, K: int) -> int:
    """Activation rows from which tq_gemm_tq1_ws transcodes an N x K matrix to TQ2."""
    r = int(lib.tq_tq1_transcode_min_m(N, K))
    _check(min(r, 0), "tq_tq1_transcode_min_m")
    return r


def tq_transcode_tq1_tq2(qs1, K: int, qs2=None, stream=None):
    """TQ2 bytes [N][K/4] (uint8, device) holding the trits of the TQ1 rows qs1 [N][ldq]."""
    import torch
    where = "tq_transcode_tq1_tq2"
    N, ldq = _rank2(qs1, "qs1", where)
    _need(qs1, "qs1", "u8", None, where)
    if qs2 is not None:
        _need(qs2, "qs2", "u8", (N, K // 4), where)
    _on_gpu(where, ("qs1", qs1), ("qs2", qs2))
    if qs2 is None:
        qs2 = torch.empty((N, K // 4), dtype=torch.uint8, device=qs1.device)
    with _device_of(qs1):
        _check(lib.tq_transcode_tq1_tq2(_ptr(qs1), ldq, N, K, _ptr(qs2),
                                        _stream(stream, qs1.device)), where)
    return qs2


def tq_gemm_tq1_ws(X, qs, scales, workspace, Y=None, stream=None):
    """tq_gemm_tq1 with a workspace (uint8 device tensor of at least N * K / 4
    bytes): from tq_tq1_transcode_min_m(N, K) rows on, the weights are
    transcoded once into it and the TQ2 kernels run."""
    where = "tq_gemm_tq1_ws"
    M, N, K, ldq = _gemm_operands(X, qs, scales, where, ldq_from_qs=True)
    nbytes = 0
    if workspace is not None:
        _need(workspace, "workspace", "u8", None, where)
        nbytes = workspace.numel()
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales), ("workspace", workspace)))
    with _device_of(X):
        _check(lib.tq_gemm_tq1_ws(_ptr(X), _ptr(qs), ldq, _ptr(scales), _ptr(Y), M, N, K,
                                  _ptr(workspace), nbytes, _stream(stream, X.device)), where)
    return Y


def tq_stream_read(src, sink, stream=None):
    """Read every byte of the contiguous device tensor src once (the practical
    read ceiling); sink is an int32 device tensor of at least one element."""
    where = "tq_stream_read"
    import torch
    if not torch.is_tensor(src):
        raise TQError(TQ_ERR_VALUE, f"{where}: src must be a torch tensor")
    if not src.is_contiguous():
        raise TQError(TQ_ERR_SHAPE, f"{where}: src must be contiguous")
    _need(sink, "sink", "i32", None, where)
    if sink.numel() < 1:
        raise TQError(TQ_ERR_SHAPE, f"{where}: sink needs at least one int32")
    _on_gpu(where, ("src", src), ("sink", sink))
    nbytes = src.numel() * src.element_size()
    with _device_of(src):
        _check(lib.tq_stream_read(_ptr(src), nbytes, _ptr(sink), _stream(stream, src.device)),
               where)


def tq_gemm_tq2_tile(X, qs, scales, mt: int, nr: int, ng: int, kg: int, Y=None, stream=None):
    """tq_gemm_tq2 on the tiled kernel with an explicit (mt, nr, ng, kg) tile."""
    where = "tq_gemm_tq2_tile"
    M, N, K, _ = _gemm_operands(X, qs, scales, where)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq2_tile(_ptr(X), _ptr(qs), _ptr(scales), _ptr(Y), M, N, K, mt, nr, ng,
                                    kg, _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq2_wide(X, qs, scales, mt: int, nt: int, ng: int, kg: int, Y=None, stream=None):
    """tq_gemm_tq2 on the wide-tile kernel with an explicit (mt, nt, ng, kg) tile."""
    where = "tq_gemm_tq2_wide"
    M, N, K, _ = _gemm_operands(X, qs, scales, where)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq2_wide(_ptr(X), _ptr(qs), _ptr(scales), _ptr(Y), M, N, K, mt, nt, ng,
                                    kg, _stream(stream, X.device)), where)
    return Y


def tq_gemm_tq1_tile(X, qs, scales, mt: int, nr: int, ng: int, kg: int, Y=None, stream=None):
    """tq_gemm_tq1 on the table-decode tiled kernel with an explicit tile."""
    where = "tq_gemm_tq1_tile"
    M, N, K, ldq = _gemm_operands(X, qs, scales, where, ldq_from_qs=True)
    Y = _out(Y, M, N, where, (("X", X), ("qs", qs), ("scales", scales)))
    with _device_of(X):
        _check(lib.tq_gemm_tq1_tile(_ptr(X), _ptr(qs), ldq, _ptr(scales), _ptr(Y), M, N, K, mt,
                                    nr, ng, kg, _stream(stream, X.device)), where)
    return Y


def tq_pack_dev(fmt: int, W, eps: float = 1e-5, ldq: int | None = None, stream=None):
    """On-device ternarize + pack of a float32 [N][K] device tensor W (fmt 2 or 1).
    Returns device tensors (qs, scales fp16, gamma fp64 [1], status int32 [1])."""
    import torch
    where = "tq_pack_tq%d_dev" % fmt
    if fmt not in (1, 2):
        raise TQError(TQ_ERR_VALUE, f"{where}: format must be 1 or 2")
    N, K = _rank2(W, "W", where)
    _need(W, "W", "f32", None, where)
    _on_gpu(where, ("W", W))
    dev = W.device
    if fmt == 2:
        qs = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
    else:
        ldq = tq_tq1_ldq(K) if ldq is None else ldq
        qs = torch.empty((N, max(ldq, 0)), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // 256), dtype=torch.float16, device=dev)
    gamma = torch.empty(1, dtype=torch.float64, device=dev)
    status = torch.empty(1, dtype=torch.int32, device=dev)
    wsb = lib.tq_pack_dev_workspace_bytes(N, K)
    if wsb < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_pack_dev_workspace_bytes")
    ws = torch.empty(int(wsb), dtype=torch.uint8, device=dev)
    with _device_of(W):
        sp = _stream(stream, dev)
        if fmt == 2:
            st = lib.tq_pack_tq2_dev(_ptr(W), N, K, float(eps), _ptr(qs), _ptr(scales),
                                     _ptr(gamma), _ptr(status), _ptr(ws), wsb, sp)
        else:
            st = lib.tq_pack_tq1_dev(_ptr(W), N, K, float(eps), ldq, _ptr(qs), _ptr(scales),
                                     _ptr(gamma), _ptr(status), _ptr(ws), wsb, sp)
    _check(st, where)
    return qs, scales, gamma, status


def tq_pack_tq2_dev_noalloc(W, qs, scales, gamma, status, eps: float = 1e-5, stream=None):
    """tq_pack_tq2_dev into caller-owned outputs with the library's fixed
    per-device workspace (no device allocation by this call): W float32
    [N][K], qs uint8 [N][K/4], scales fp16 [N][K/256], gamma float64 [1],
    status int32 [1], all on one GPU."""
    import torch
    where = "tq_pack_tq2_dev_noalloc"
    N, K = _rank2(W, "W", where)
    _need(W, "W", "f32", None, where)
    _need(qs, "qs", "u8", (N, K // 4), where)
    _need(scales, "scales", "f16", (N, K // 256), where)
    if not (torch.is_tensor(gamma) and gamma.dtype == torch.float64 and gamma.numel() >= 1):
        raise TQError(TQ_ERR_VALUE, f"{where}: gamma must be a float64 tensor of >= 1 element")
    if not (torch.is_tensor(status) and status.dtype == torch.int32 and status.numel() >= 1):
        raise TQError(TQ_ERR_VALUE, f"{where}: status must be an int32 tensor of >= 1 element")
    _on_gpu(where, ("W", W), ("qs", qs), ("scales", scales), ("gamma", gamma), ("status", status))
    with _device_of(W):
        _check(lib.tq_pack_tq2_dev_noalloc(_ptr(W), N, K, float(eps), _ptr(qs), _ptr(scales),
                                           _ptr(gamma), _ptr(status), _stream(stream, W.device)),
               where)


def tq_gemm_tq2(X, qs, scales, Y=None, stream=None):
    return tq_gemm_tq2_ex(X, qs, scales, TQ_PATH_AUTO, Y, stream)


def tq_gemm_tq1(X, qs, scales, Y=None, stream=None):
    return tq_gemm_tq1_ex(X, qs, scales, TQ_PATH_AUTO, Y, stream)


def tq_kernel_name(fmt: int, M: int, N: int, K: int, path: int = TQ_PATH_AUTO) -> str:
    """Kernel that the product with this format (2 or 1), shape and path runs."""
    buf = C.create_string_buffer(128)
    _check(lib.tq_kernel_name(fmt, M, N, K, path, buf, 128), "tq_kernel_name")
    return buf.value.decode()


# ------------------------------------------------------------------ decode
#
# These calls are a few microseconds of GPU work in a decode step: the common form
# of each is compiled (_fast), and the functions here say what is wrong with any
# other, or serve outputs, workspaces and streams that the caller brings.

if _torch is not None:
    _KIND = {_torch.float16: TQ_F16, _torch.bfloat16: TQ_BF16, _torch.float32: TQ_F32}
    _I32T = _torch.int32


def _kind(t, name, where, f32=False):
    """tq_dtype of a float tensor."""
    if not isinstance(t, _torch.Tensor):
        raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be a torch tensor")
    k = _KIND.get(t.dtype)
    if k is None or (k == TQ_F32 and not f32):
        raise TQError(TQ_ERR_VALUE, f"{where}: {name} has dtype {t.dtype}")
    return k


def _flag(v, name, where):
    """A bool, or 0 or 1, as an int."""
    try:
        if v == 0 or v == 1:
            return int(v)
    except (RuntimeError, TypeError, ValueError):  # an array or a tensor of several
        pass
    raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be True or False, not {v!r}")


def _heads(t, name, where):
    """Shape and strides of a [tokens][heads][D] tensor, the numbers of a head adjacent."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or (strides[2] != 1 and shape[2] > 1):
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be [tokens][heads][D] with adjacent "
                                    f"numbers, not {tuple(shape)} at strides {strides}")
    return shape, strides


def _same(t, name, like, shape, where, strided=False):
    """An output of the type and shape of another tensor's."""
    if not isinstance(t, _torch.Tensor) or t.dtype != like.dtype:
        raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be a tensor of {like.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} has shape {tuple(t.shape)}, "
                                    f"expected {tuple(shape)}")
    if strided:
        _heads(t, name, where)
    elif not t.is_contiguous():
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be contiguous (row-major)")


def _int32(t, name, shape, where):
    """An int32 tensor of the given shape, contiguous."""
    if not (isinstance(t, _torch.Tensor) and t.dtype is _I32T and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, "i32", shape, where)


def _cache(k_pages, v_pages, like, D, where):
    """(n_pages, page_size, Hkv, page, row and head stride) of the two halves of a
    paged cache [pages][slots][Hkv][D], any order in memory, numbers adjacent."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, _torch.Tensor):
            raise TQError(TQ_ERR_VALUE, f"{where}: {name} must be a torch tensor")
    ks, kst = k_pages.shape, k_pages.stride()
    if not (k_pages.dtype is v_pages.dtype is like.dtype and len(ks) == 4 and ks[3] == D
            and kst[3] == 1 and v_pages.shape == ks and v_pages.stride() == kst):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.dtype != like.dtype:
                raise TQError(TQ_ERR_VALUE, f"{where}: {name} is {t.dtype}, expected {like.dtype}")
            if t.dim() != 4 or t.shape[3] != D or (D > 1 and t.stride(3) != 1):
                raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be [pages][slots][heads][{D}] "
                                            f"with adjacent numbers, not {tuple(t.shape)}")
        if v_pages.shape != ks or v_pages.stride() != kst:
            raise TQError(TQ_ERR_SHAPE, f"{where}: k_pages and v_pages differ in shape or strides")
    return ks[0], ks[1], ks[2], kst[0], kst[1], kst[2]


def _table(table, where):
    """(n_pos, rot) of a cosine / sine table [n_pos][rot / 2][2]."""
    shape = table.shape if isinstance(table, _torch.Tensor) else ()
    if len(shape) != 3 or shape[2] != 2:
        raise TQError(TQ_ERR_SHAPE, f"{where}: table must be [positions][rot / 2][2]")
    if table.dtype is not _torch.float32 or not table.is_contiguous():
        _need(table, "table", "f32", None, where)
    return shape[0], 2 * shape[1]


def _rows(t, name, where):
    """(rows, width) of a contiguous int32 matrix."""
    shape = t.shape if isinstance(t, _torch.Tensor) else ()
    if len(shape) != 2:
        raise TQError(TQ_ERR_SHAPE, f"{where}: {name} must be a 2-D tensor")
    if t.dtype is not _I32T or not t.is_contiguous():
        _need(t, name, "i32", None, where)
    return shape


def _empty(like, shape, dtype, stream):
    """A new tensor on like's GPU whose memory belongs to the stream that the call
    runs on: the allocator hands a freed block out again in the order of its own
    stream, so memory of the current stream must not be written on another one."""
    device = like.device
    if stream is None or stream == _torch._C._cuda_getCurrentRawStream(device.index):
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(_torch.cuda.default_stream(device) if stream == 0 else
                            _torch.cuda.ExternalStream(stream, device)):
        return _torch.empty(shape, dtype=dtype, device=device)


def _pieces(like, sizes, stream):
    """int32 vectors of the given sizes from one allocation."""
    return _empty(like, (sum(sizes),), _I32T, stream).split_with_sizes(sizes)


def _done(r, where):
    """The result of a compiled call, or TQError for its status."""
    if type(r) is int:
        raise TQError(r, where)
    return r


def _launch(where, dev, fn, *args):
    """Call a C entry point with GPU `dev` current and raise for its status."""
    if _torch.cuda.current_device() != dev:
        with _torch.cuda.device(dev):
            st = fn(*args)
    else:
        st = fn(*args)
    if st:
        raise TQError(st, where)


def _raw_stream(stream, dev):
    if stream is not None:
        return stream
    return _torch._C._cuda_getCurrentRawStream(dev)


def tq_rope_table(n_pos: int, rot: int, theta: float = 5e5, scaling: int = TQ_ROPE_NONE,
                  factor: float = 1.0, trained: float = 4096.0, fast: float = 32.0,
                  slow: float = 1.0, gain: float = 1.0) -> np.ndarray:
    """Cosines and sines float32 [n_pos][rot / 2][2] (numpy) for tq_rope."""
    table = np.empty((max(n_pos, 0), max(rot // 2, 0), 2), dtype=np.float32)
    _check(lib.tq_rope_table(n_pos, rot, theta, scaling, factor, trained, fast, slow, gain,
                             _ptr(table)), "tq_rope_table")
    return table


def tq_rope(X, table, positions, interleaved: bool = False, inverse: bool = False, Y=None,
            stream=None):
    """Rotary positions: X [T][H][D] (fp16, bfloat16 or float32; a view with any
    strides, numbers of a head adjacent) turned by table[positions] over the first
    rot numbers of each head; inverse turns back, which is the gradient.  Y may be
    X; a new contiguous tensor when None.  Like every call here it is unknown to
    autograd: the result of an X that requires a gradient requires none, and a
    torch.autograd.Function that is to carry one calls this with inverse in its
    backward."""
    where = "tq_rope"
    if Y is None and stream is None:
        r = _fast.rope(X, table, positions, interleaved, inverse)
        if r is not None:
            return _done(r, where)
    kind = _kind(X, "X", where, f32=True)
    interleaved, inverse = _flag(interleaved, "interleaved", where), _flag(inverse, "inverse", where)
    (T, H, D), xs = _heads(X, "X", where)
    n_pos, rot = _table(table, where)
    _int32(positions, "positions", (T,), where)
    if Y is not None:
        _same(Y, "Y", X, (T, H, D), where, strided=True)
    dev = X.get_device()
    if dev < 0 or table.get_device() != dev or positions.get_device() != dev or (
            Y is not None and Y.get_device() != dev):
        _on_gpu(where, ("X", X), ("table", table), ("positions", positions), ("Y", Y))
    if Y is None:
        Y = _empty(X, (T, H, D), X.dtype, stream)
    ys = Y.stride()
    _launch(where, dev, lib.tq_rope, kind, X.data_ptr(), xs[0], xs[1], Y.data_ptr(), ys[0], ys[1],
            table.data_ptr(), n_pos, rot, positions.data_ptr(), T, H, D, interleaved, inverse,
            _raw_stream(stream, dev))
    return Y


def tq_rope_append(QKV, table, positions, page_table, k_pages, v_pages, interleaved: bool = False,
                   seqs=None, Q=None, stream=None):
    """Rotate the query and key heads of QKV [T][Hq + 2 Hkv][D], write the keys and
    values of token t into slot positions[t] of row seqs[t] (t when None) of the
    paged cache, and return the queries [T][Hq][D].  k_pages, v_pages:
    [pages][slots][Hkv][D], any strides, numbers of a head adjacent."""
    where = "tq_rope_append"
    if Q is None and stream is None:
        r = _fast.rope_append(QKV, table, positions, page_table, k_pages, v_pages, interleaved,
                              seqs)
        if r is not None:
            return _done(r, where)
    kind = _kind(QKV, "QKV", where)
    interleaved = _flag(interleaved, "interleaved", where)
    (T, H, D), xs = _heads(QKV, "QKV", where)
    if H > 1 and xs[1] != D:
        raise TQError(TQ_ERR_SHAPE, f"{where}: the heads of QKV must be adjacent")
    n_pos, rot = _table(table, where)
    _int32(positions, "positions", (T,), where)
    n_seqs, width = _rows(page_table, "page_table", where)
    if seqs is not None:
        _int32(seqs, "seqs", (T,), where)
    P, size, Hkv, page_stride, row_stride, head_stride = _cache(k_pages, v_pages, QKV, D, where)
    Hq = H - 2 * Hkv
    if Hq < 1:
        raise TQError(TQ_ERR_SHAPE, f"{where}: {H} heads in QKV, {Hkv} in the cache")
    if Q is not None:
        _same(Q, "Q", QKV, (T, Hq, D), where)
    dev = QKV.get_device()
    if dev < 0 or not (table.get_device() == positions.get_device() == page_table.get_device()
                       == k_pages.get_device() == v_pages.get_device() == dev) or (
            seqs is not None and seqs.get_device() != dev) or (
            Q is not None and Q.get_device() != dev):
        _on_gpu(where, ("QKV", QKV), ("table", table), ("positions", positions),
                ("page_table", page_table), ("seqs", seqs), ("k_pages", k_pages),
                ("v_pages", v_pages), ("Q", Q))
    if Q is None:
        Q = _empty(QKV, (T, Hq, D), QKV.dtype, stream)
    _launch(where, dev, lib.tq_rope_append, kind, QKV.data_ptr(), xs[0], table.data_ptr(), n_pos,
            rot, positions.data_ptr(), None if seqs is None else seqs.data_ptr(),
            page_table.data_ptr(), n_seqs, width, k_pages.data_ptr(), v_pages.data_ptr(), P, size,
            page_stride, row_stride, head_stride, Q.data_ptr(), T, Hq, Hkv, D, interleaved,
            _raw_stream(stream, dev))
    return Q


def tq_paged_attention_workspace(B: int, Hq: int, Hkv: int, D: int, page_size: int,
                                 width: int) -> int:
    """Workspace bytes of tq_paged_attention on the current GPU."""
    n = int(lib.tq_paged_attention_workspace(B, Hq, Hkv, D, page_size, width))
    _check(min(n, 0), "tq_paged_attention_workspace")
    return n


@functools.lru_cache(maxsize=256)
def _attention_workspace(dev, *shape):
    with _torch.cuda.device(dev):  # the size follows the GPU's compute units
        return lib.tq_paged_attention_workspace(*shape)


def tq_paged_attention(Q, k_pages, v_pages, page_table, lens, scale: float | None = None,
                       window: int = 0, out=None, return_lse: bool = False, workspace=None,
                       stream=None):
    """Attention of one new token per sequence: Q [B][Hq][D] over the last `window`
    (0: all) of lens[b] tokens in the paged cache k_pages, v_pages
    [pages][slots][Hkv][D] named by page_table [B][width].  Returns out [B][Hq][D],
    and lse float32 [B][Hq] with return_lse.  scale: 1 / sqrt(D) when None."""
    where = "tq_paged_attention"
    if out is None and workspace is None and stream is None:
        r = _fast.paged_attention(Q, k_pages, v_pages, page_table, lens, scale, window, return_lse)
        if r is not None:
            return _done(r, where)
    kind = _kind(Q, "Q", where)
    (B, Hq, D), qs = _heads(Q, "Q", where)
    P, size, Hkv, page_stride, row_stride, head_stride = _cache(k_pages, v_pages, Q, D, where)
    rows, width = _rows(page_table, "page_table", where)
    if rows != B:
        raise TQError(TQ_ERR_SHAPE, f"{where}: page_table has {rows} rows, Q {B}")
    _int32(lens, "lens", (B,), where)
    if out is not None:
        _same(out, "out", Q, (B, Hq, D), where)
    if workspace is not None:
        _need(workspace, "workspace", "u8", None, where)
    dev = Q.get_device()
    if dev < 0 or not (k_pages.get_device() == v_pages.get_device() == page_table.get_device()
                       == lens.get_device() == dev) or (
            out is not None and out.get_device() != dev) or (
            workspace is not None and workspace.get_device() != dev):
        _on_gpu(where, ("Q", Q), ("k_pages", k_pages), ("v_pages", v_pages),
                ("page_table", page_table), ("lens", lens), ("out", out),
                ("workspace", workspace))
    if workspace is None:
        n = _attention_workspace(dev, B, Hq, Hkv, D, size, width)
        if n:
            _check(min(n, 0), where)
            workspace = _empty(Q, (n,), _torch.uint8, stream)
    else:
        n = workspace.numel()
    if out is None:
        out = _empty(Q, (B, Hq, D), Q.dtype, stream)
    lse = _empty(Q, (B, Hq), _torch.float32, stream) if return_lse else None
    _launch(where, dev, lib.tq_paged_attention, kind, Q.data_ptr(), qs[0], qs[1],
            k_pages.data_ptr(), v_pages.data_ptr(), P, size, page_stride, row_stride, head_stride,
            page_table.data_ptr(), width, lens.data_ptr(), B, Hq, Hkv, D,
            1.0 / math.sqrt(D) if scale is None else scale, window, out.data_ptr(),
            None if lse is None else lse.data_ptr(),
            None if workspace is None else workspace.data_ptr(), n, _raw_stream(stream, dev))
    return (out, lse) if return_lse else out


def _pool(pool, where):
    """(planes, n_pages, bytes of a page) of a contiguous pool [planes][pages]..."""
    if not isinstance(pool, _torch.Tensor) or pool.dim() < 3 or not pool.is_contiguous():
        raise TQError(TQ_ERR_SHAPE, f"{where}: pool must be a contiguous [planes][pages][...] tensor")
    size = pool.element_size()
    for n in pool.shape[2:]:
        size *= n
    return pool.shape[0], pool.shape[1], size


def _state(page_table, lens, where):
    rows, width = _rows(page_table, "page_table", where)
    _int32(lens, "lens", (rows,), where)
    return rows, width


@functools.lru_cache(maxsize=256)
def tq_pages_workspace(rows: int, n_pages: int) -> int:
    """Workspace bytes of tq_pages_fork, tq_pages_grow and tq_pages_compact."""
    n = int(lib.tq_pages_workspace(rows, n_pages))
    _check(min(n, 0), "tq_pages_workspace")
    return n


def tq_pages_fork(pool, page_table, lens, parent, page_size: int, stream=None):
    """Continue row parent[r] as row r (an empty sequence where parent[r] names no
    row): pages are shared, a partly filled last page is copied for all but the
    first row that continues it.  pool [planes][pages][...], page_table [rows][width],
    lens [rows], parent [new rows].  Returns (page_table, lens, refs, short): the new
    state, how often each page is held, and the rows that found no free page."""
    where = "tq_pages_fork"
    if stream is None:
        r = _fast.pages_fork(pool, page_table, lens, parent, page_size)
        if r is not None:
            return _done(r, where)
    planes, P, size = _pool(pool, where)
    rows_in, width = _state(page_table, lens, where)
    if not isinstance(parent, _torch.Tensor) or parent.dim() != 1:
        raise TQError(TQ_ERR_SHAPE, f"{where}: parent must be a 1-D tensor")
    rows = parent.shape[0]
    _int32(parent, "parent", (rows,), where)
    dev = pool.get_device()
    if dev < 0 or not (page_table.get_device() == lens.get_device() == parent.get_device() == dev):
        _on_gpu(where, ("pool", pool), ("page_table", page_table), ("lens", lens),
                ("parent", parent))
    n = tq_pages_workspace(rows, P)
    ws, table_out, lens_out, refs, short = _pieces(lens, (n // 4, rows * width, rows, P, 1), stream)
    _launch(where, dev, lib.tq_pages_fork, pool.data_ptr(), planes, P, size, page_table.data_ptr(),
            lens.data_ptr(), rows_in, parent.data_ptr(), rows, width, page_size,
            table_out.data_ptr(), lens_out.data_ptr(), refs.data_ptr(), short.data_ptr(),
            ws.data_ptr(), n, _raw_stream(stream, dev))
    return table_out.view(rows, width), lens_out, refs, short


def tq_pages_grow(page_table, lens, add, n_pages: int, page_size: int, stream=None):
    """Room for add[r] more tokens in row r, from the pages that no row holds.
    Returns (page_table, lens, short): the new state and how many rows were refused."""
    where = "tq_pages_grow"
    if stream is None:
        r = _fast.pages_grow(page_table, lens, add, n_pages, page_size)
        if r is not None:
            return _done(r, where)
    rows, width = _state(page_table, lens, where)
    _int32(add, "add", (rows,), where)
    dev = page_table.get_device()
    if dev < 0 or not (lens.get_device() == add.get_device() == dev):
        _on_gpu(where, ("page_table", page_table), ("lens", lens), ("add", add))
    n = tq_pages_workspace(rows, n_pages)
    ws, table_out, lens_out, short = _pieces(lens, (n // 4, rows * width, rows, 1), stream)
    _launch(where, dev, lib.tq_pages_grow, page_table.data_ptr(), lens.data_ptr(), add.data_ptr(),
            rows, width, page_size, n_pages, table_out.data_ptr(), lens_out.data_ptr(),
            short.data_ptr(), ws.data_ptr(), n, _raw_stream(stream, dev))
    return table_out.view(rows, width), lens_out, short


def tq_pages_compact(pool, page_table, lens, page_size: int, stream=None):
    """Move the pages in use to the low end of the pool.  Returns (page_table, used):
    the new table and the number of pages in use (int32 [1]), all below it."""
    where = "tq_pages_compact"
    if stream is None:
        r = _fast.pages_compact(pool, page_table, lens, page_size)
        if r is not None:
            return _done(r, where)
    planes, P, size = _pool(pool, where)
    rows, width = _state(page_table, lens, where)
    dev = pool.get_device()
    if dev < 0 or not (page_table.get_device() == lens.get_device() == dev):
        _on_gpu(where, ("pool", pool), ("page_table", page_table), ("lens", lens))
    n = tq_pages_workspace(rows, P)
    ws, table_out, used = _pieces(lens, (n // 4, rows * width, 1), stream)
    _launch(where, dev, lib.tq_pages_compact, pool.data_ptr(), planes, P, size,
            page_table.data_ptr(), lens.data_ptr(), rows, width, page_size, table_out.data_ptr(),
            used.data_ptr(), ws.data_ptr(), n, _raw_stream(stream, dev))
    return table_out.view(rows, width), used


def tq_pages_copy(pool, src, dst, stream=None):
    """Copy page src[i] over page dst[i] in every plane of pool [planes][pages][...]."""
    where = "tq_pages_copy"
    planes, P, size = _pool(pool, where)
    if not isinstance(src, _torch.Tensor) or src.dim() != 1:
        raise TQError(TQ_ERR_SHAPE, f"{where}: src must be a 1-D tensor")
    _int32(src, "src", src.shape, where)
    _int32(dst, "dst", src.shape, where)
    dev = pool.get_device()
    if dev < 0 or not (src.get_device() == dst.get_device() == dev):
        _on_gpu(where, ("pool", pool), ("src", src), ("dst", dst))
    _launch(where, dev, lib.tq_pages_copy, pool.data_ptr(), planes, P, size, src.data_ptr(),
            dst.data_ptr(), src.shape[0], _raw_stream(stream, dev))


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw arguments and return its status (for tests)."""
    return getattr(lib, name)(*args)
