"""Python binding of the GB300 persistent batched GEMM with fused epilogue.

Thin ctypes layer over ``libgemm_gb300.so`` (C ABI in ``include/gemm_gb300.h``):
the functions below carry the C entry points' names and only marshal
arguments.  Every step of the computation runs in the library's CUDA kernel;
there is no fallback, and a missing library raises immediately.

    Y = A*B,   D = alpha*(A*B) + beta*C + x_factor*X

Tensor arguments may be raw device addresses (int) or objects with a
``data_ptr()`` method (e.g. torch CUDA tensors); streams may be an int handle
or an object with a ``cuda_stream`` attribute.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
# The library for a process that drives one GPU (every kernel variant), and
# the one for processes that drive several GPUs (no multicast kernels).
LIB_PATH = os.path.join(_HERE, "libgemm_gb300.so")
NOMC_LIB_PATH = os.path.join(_HERE, "libgemm_gb300_nomc.so")

# enums (include/gemm_gb300.h)
GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED_DTYPE = 2
GEMM_ERR_MISALIGNED = 3
GEMM_ERR_UNSUPPORTED_ARCH = 4
GEMM_ERR_CUDA = 5
GEMM_ERR_DEVICE_TIMEOUT = 6
GEMM_ERR_UNSUPPORTED_CONFIG = 7
GEMM_ERR_DEVICE_CHECK = 8

GEMM_F32, GEMM_F16, GEMM_BF16, GEMM_E4M3, GEMM_E5M2, GEMM_TF32 = 0, 1, 2, 3, 4, 5
GEMM_K_MAJOR, GEMM_MN_MAJOR = 0, 1
GEMM_EPI_LINEAR, GEMM_EPI_RELU = 0, 1
GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_TANH, GEMM_ACT_SILU = 0, 1, 2, 3, 4
GEMM_RING_STAT_WORDS = 16

DTYPE_CODES = {"f32": GEMM_F32, "f16": GEMM_F16, "bf16": GEMM_BF16, "e4m3": GEMM_E4M3,
               "e5m2": GEMM_E5M2, "tf32": GEMM_TF32}


ACTIVATION_CODES = {None: GEMM_ACT_NONE, "none": GEMM_ACT_NONE, "relu": GEMM_ACT_RELU,
                    "gelu": GEMM_ACT_GELU, "gelu_tanh": GEMM_ACT_GELU_TANH,
                    "silu": GEMM_ACT_SILU}


class gemm_dtypes_t(ctypes.Structure):
    _fields_ = [("ab", ctypes.c_int), ("c", ctypes.c_int), ("d", ctypes.c_int),
                ("x", ctypes.c_int), ("y", ctypes.c_int), ("cdxy_major", ctypes.c_int),
                ("b", ctypes.c_int), ("epilogue", ctypes.c_int), ("acc", ctypes.c_int)]


class gemm_config_t(ctypes.Structure):
    _fields_ = [("cta_group", ctypes.c_int), ("tile_n", ctypes.c_int), ("stages", ctypes.c_int),
                ("group_m", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_k", ctypes.c_int),
                ("acc_stages", ctypes.c_int), ("ring_bytes", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("tiles", ctypes.c_int64),
                ("grid_ctas", ctypes.c_int), ("epi_slots", ctypes.c_int),
                ("epi_slot_bytes", ctypes.c_int), ("cluster_m", ctypes.c_int),
                ("l2_hints", ctypes.c_int), ("epi_wait_ns", ctypes.c_int),
                ("inject_stall", ctypes.c_int), ("tail_split", ctypes.c_int),
                ("cluster_n", ctypes.c_int),
                ("epi_warps", ctypes.c_int),
                ("stream_k", ctypes.c_int),
                ("split_k", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class gemm_problem_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("L", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("layoutA", ctypes.c_int),
                ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("layoutB", ctypes.c_int),
                ("C", ctypes.c_void_p), ("X", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("Y", ctypes.c_void_p),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("x_factor", ctypes.c_float),
                ("dtypes", gemm_dtypes_t)]


class gemm_rmsnorm_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("H", ctypes.c_int64),
                ("type", ctypes.c_int), ("w_type", ctypes.c_int), ("y_type", ctypes.c_int),
                ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("r", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class gemm_rmsnorm_bwd_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("H", ctypes.c_int64),
                ("type", ctypes.c_int), ("w_type", ctypes.c_int), ("dw_type", ctypes.c_int),
                ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dweight", ctypes.c_void_p)]


class gemm_linear_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_type", ctypes.c_int), ("b_type", ctypes.c_int), ("bias_type", ctypes.c_int),
                ("r_type", ctypes.c_int), ("z_type", ctypes.c_int), ("d_type", ctypes.c_int),
                ("layoutA", ctypes.c_int), ("layoutB", ctypes.c_int),
                ("activation", ctypes.c_int), ("alpha", ctypes.c_float),
                ("A", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("row_scale", ctypes.c_void_p), ("col_scale", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("R", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("Z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("D", ctypes.c_void_p), ("ldd", ctypes.c_int64)]


class gemm_linear_bwd_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("type", ctypes.c_int), ("da_type", ctypes.c_int), ("db_type", ctypes.c_int),
                ("dbias_type", ctypes.c_int), ("activation", ctypes.c_int),
                ("accumulate", ctypes.c_int), ("alpha", ctypes.c_float),
                ("dd", ctypes.c_void_p), ("lddd", ctypes.c_int64),
                ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("a", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("dz", ctypes.c_void_p), ("lddz", ctypes.c_int64),
                ("da", ctypes.c_void_p), ("ldda", ctypes.c_int64),
                ("db", ctypes.c_void_p), ("lddb", ctypes.c_int64), ("dbias", ctypes.c_void_p)]


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {gemm_status_string(status)}" if what else
                         gemm_status_string(status))


_lock = threading.Lock()
_lib = None


def select_library(path: str) -> None:
    """Load the library at `path` instead of the product one (the
    ring-statistics build, for instance).  Must precede the first call."""
    global LIB_PATH
    with _lock:
        if _lib is not None and os.path.abspath(path) != os.path.abspath(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is already loaded")
        LIB_PATH = path


def library():
    """Load libgemm_gb300.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(LIB_PATH)
            i32, i64, f32, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
            lib.gemm_create.argtypes = [ctypes.POINTER(vp), i32]
            lib.gemm_destroy.argtypes = [vp]
            lib.gemm_run.argtypes = [vp, i64, i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, vp,
                                     vp, vp, f32, f32, f32, ctypes.POINTER(gemm_dtypes_t), vp]
            lib.gemm_run_host.argtypes = list(lib.gemm_run.argtypes)
            lib.gemm_ring_stats.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint64), i32,
                                            ctypes.POINTER(ctypes.c_int)]
            lib.gemm_sync_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
            lib.gemm_run_noalloc.argtypes = [i64, i64, i64, i64, vp, i64, i32, vp, i64, i32, vp,
                                             vp, vp, vp, f32, f32, f32,
                                             ctypes.POINTER(gemm_dtypes_t), vp,
                                             ctypes.POINTER(ctypes.c_uint32)]
            lib.gemm_status_string.argtypes = [i32]
            lib.gemm_status_string.restype = ctypes.c_char_p
            lib.gemm_check.argtypes = [ctypes.POINTER(gemm_problem_t)]
            lib.gemm_plan.argtypes = [ctypes.POINTER(gemm_problem_t), i32, i32,
                                      ctypes.POINTER(gemm_config_t), ctypes.POINTER(gemm_config_t)]
            lib.gemm_set_config.argtypes = [vp, ctypes.POINTER(gemm_config_t)]
            lib.gemm_last_config.argtypes = [vp, ctypes.POINTER(gemm_config_t)]
            lib.gemm_tmem_columns.argtypes = [i32, i32]
            lib.gemm_set_timeout_ns.argtypes = [vp, ctypes.c_uint64]
            lib.gemm_rmsnorm.argtypes = [vp, vp, vp]
            lib.gemm_rmsnorm_check.argtypes = [ctypes.POINTER(gemm_rmsnorm_t)]
            lib.gemm_rmsnorm_bwd_check.argtypes = [ctypes.POINTER(gemm_rmsnorm_bwd_t)]
            lib.gemm_rmsnorm_bwd_workspace.argtypes = [i64, i64]
            lib.gemm_rmsnorm_bwd_workspace.restype = i64
            lib.gemm_rmsnorm_bwd.argtypes = [vp, vp, vp, i64, vp]
            lib.gemm_linear_check.argtypes = [ctypes.POINTER(gemm_linear_t)]
            lib.gemm_linear.argtypes = [vp, vp, vp]
            lib.gemm_linear_bwd_check.argtypes = [ctypes.POINTER(gemm_linear_bwd_t)]
            lib.gemm_linear_bwd.argtypes = [vp, vp, vp]
            for name in ("gemm_create", "gemm_destroy", "gemm_run", "gemm_run_noalloc",
                         "gemm_sync_status",
                         "gemm_check", "gemm_plan", "gemm_set_config", "gemm_last_config",
                         "gemm_tmem_columns", "gemm_set_timeout_ns", "gemm_rmsnorm",
                         "gemm_rmsnorm_check", "gemm_rmsnorm_bwd", "gemm_rmsnorm_bwd_check",
                         "gemm_linear", "gemm_linear_check", "gemm_linear_bwd",
                         "gemm_linear_bwd_check"):
                getattr(lib, name).restype = i32
            _lib = lib
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t or None
    return int(t.data_ptr())


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s or None
    return int(s.cuda_stream)


def make_dtypes(ab, c="f32", d="f32", x="f32", y="f32", cdxy_major=GEMM_K_MAJOR, b=None,
                epilogue=GEMM_EPI_LINEAR, acc="f32") -> gemm_dtypes_t:
    """b: B's type when it differs from A's (fp8 pairs); epilogue: GEMM_EPI_*;
    acc: the tensor-core accumulator type, "f32" or "f16"."""
    code = lambda v: DTYPE_CODES[v] if isinstance(v, str) else int(v)
    return gemm_dtypes_t(code(ab), code(c), code(d), code(x), code(y), int(cdxy_major),
                         GEMM_F32 if b is None or b == ab else code(b), int(epilogue), code(acc))


# ------------------------------------------------------------------ C entry points

def gemm_status_string(status: int) -> str:
    return library().gemm_status_string(int(status)).decode()


def gemm_create(device: int = 0) -> int:
    h = ctypes.c_void_p()
    st = library().gemm_create(ctypes.byref(h), int(device))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_create")
    return h.value


def gemm_destroy(handle: int) -> None:
    st = library().gemm_destroy(handle)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_destroy")


def gemm_run(handle, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y,
             alpha, beta, x_factor, dtypes: gemm_dtypes_t, stream=None, check=True) -> int:
    st = library().gemm_run(handle, M, N, K, L, _ptr(A), lda, layoutA, _ptr(B), ldb, layoutB,
                            _ptr(C), _ptr(X), _ptr(D), _ptr(Y), alpha, beta, x_factor,
                            ctypes.byref(dtypes), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_run")
    return st


def gemm_run_host(handle, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y,
                  alpha, beta, x_factor, dtypes: gemm_dtypes_t, stream=None,
                  check=True) -> int:
    """gemm_run on HOST buffers (CPU tensors, pinned for overlap): the library
    copies the inputs in, runs the GEMM and copies D and Y back, all enqueued
    on `stream` (see the C header)."""
    st = library().gemm_run_host(handle, M, N, K, L, _ptr(A), lda, layoutA, _ptr(B), ldb,
                                 layoutB, _ptr(C), _ptr(X), _ptr(D), _ptr(Y), alpha, beta,
                                 x_factor, ctypes.byref(dtypes), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_run_host")
    return st


def gemm_run_noalloc(M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y, alpha, beta,
                     x_factor, dtypes: gemm_dtypes_t, stream=None, check=True,
                     watchdog=False) -> tuple[int, int]:
    """gemm_run without a handle and without allocating device memory (the
    watchdog status word lives in a static device array); see the C header.
    watchdog=True makes the call synchronise and report the status word.
    Returns (status, watchdog word)."""
    word = ctypes.c_uint32(0)
    st = library().gemm_run_noalloc(M, N, K, L, _ptr(A), lda, layoutA, _ptr(B), ldb, layoutB,
                                    _ptr(C), _ptr(X), _ptr(D), _ptr(Y), alpha, beta, x_factor,
                                    ctypes.byref(dtypes), _stream(stream),
                                    ctypes.byref(word) if watchdog else None)
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_run_noalloc")
    return st, word.value


def gemm_sync_status(handle, stream=None) -> tuple[int, int]:
    detail = ctypes.c_uint32(0)
    st = library().gemm_sync_status(handle, _stream(stream), ctypes.byref(detail))
    return st, detail.value


def gemm_check(problem: gemm_problem_t) -> int:
    return library().gemm_check(ctypes.byref(problem))


def gemm_plan(problem: gemm_problem_t, sm_count: int, smem_optin: int,
              forced: gemm_config_t | None = None) -> tuple[int, gemm_config_t]:
    out = gemm_config_t()
    st = library().gemm_plan(ctypes.byref(problem), sm_count, smem_optin,
                             ctypes.byref(forced) if forced is not None else None,
                             ctypes.byref(out))
    return st, out


def gemm_set_config(handle, cfg: gemm_config_t | None) -> None:
    st = library().gemm_set_config(handle, ctypes.byref(cfg) if cfg is not None else None)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_set_config")


def gemm_last_config(handle) -> gemm_config_t:
    out = gemm_config_t()
    st = library().gemm_last_config(handle, ctypes.byref(out))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_last_config")
    return out


def gemm_tmem_columns(tile_m: int, tile_n: int) -> int:
    return library().gemm_tmem_columns(tile_m, tile_n)


def gemm_set_timeout_ns(handle, ns: int) -> None:
    st = library().gemm_set_timeout_ns(handle, int(ns))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_set_timeout_ns")


def make_problem(M, N, K, L, A=None, lda=0, layoutA=GEMM_K_MAJOR, B=None, ldb=0,
                 layoutB=GEMM_K_MAJOR, C=None, X=None, D=None, Y=None, alpha=1.0, beta=0.0,
                 x_factor=0.0, dtypes: gemm_dtypes_t | None = None) -> gemm_problem_t:
    """A gemm_problem_t for the host-only calls (pointers may be plain ints)."""
    return gemm_problem_t(M, N, K, L, _ptr(A), lda, layoutA, _ptr(B), ldb, layoutB, _ptr(C),
                          _ptr(X), _ptr(D), _ptr(Y), alpha, beta, x_factor,
                          dtypes if dtypes is not None else make_dtypes("f16"))


def gemm_rmsnorm(handle, problem: gemm_rmsnorm_t, stream=None, check=True) -> int:
    st = library().gemm_rmsnorm(handle, ctypes.byref(problem), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_rmsnorm")
    return st


def gemm_rmsnorm_check(problem: gemm_rmsnorm_t) -> int:
    return library().gemm_rmsnorm_check(ctypes.byref(problem))


def gemm_rmsnorm_bwd_check(problem: gemm_rmsnorm_bwd_t) -> int:
    return library().gemm_rmsnorm_bwd_check(ctypes.byref(problem))


def gemm_rmsnorm_bwd_workspace(M, H) -> int:
    """Bytes of workspace gemm_rmsnorm_bwd needs."""
    return library().gemm_rmsnorm_bwd_workspace(M, H)


def gemm_rmsnorm_bwd(handle, problem: gemm_rmsnorm_bwd_t, workspace=None, workspace_bytes=0,
                     stream=None, check=True) -> int:
    st = library().gemm_rmsnorm_bwd(handle, ctypes.byref(problem), _ptr(workspace),
                                    workspace_bytes, _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_rmsnorm_bwd")
    return st


def gemm_linear_check(problem: gemm_linear_t) -> int:
    return library().gemm_linear_check(ctypes.byref(problem))


def gemm_linear(handle, problem: gemm_linear_t, stream=None, check=True) -> int:
    st = library().gemm_linear(handle, ctypes.byref(problem), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_linear")
    return st


def gemm_linear_bwd_check(problem: gemm_linear_bwd_t) -> int:
    return library().gemm_linear_bwd_check(ctypes.byref(problem))


def gemm_linear_bwd(handle, problem: gemm_linear_bwd_t, stream=None, check=True) -> int:
    st = library().gemm_linear_bwd(handle, ctypes.byref(problem), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_linear_bwd")
    return st


# ------------------------------------------------------------------ tensors
#
# The calls on tensors fill the C structures by struct.pack (the fields of the
# ctypes structures above, in order): a call then costs about half of what building
# a ctypes structure and keyword checks would.

_RMSNORM = struct.Struct("<2q3if11Q")
_RMSNORM_BWD = struct.Struct("<2q3i4x11Q")
_LINEAR = struct.Struct("<3q9if13Q")
_LINEAR_BWD = struct.Struct("<3q6if4x15Q")

# Type codes by the name of a tensor's dtype.
_TENSOR_CODES = {"torch.float32": GEMM_F32, "torch.float16": GEMM_F16,
                 "torch.bfloat16": GEMM_BF16, "torch.float8_e4m3fn": GEMM_E4M3,
                 "torch.float8_e5m2": GEMM_E5M2}
_CODE_OF = {}           # the same by the dtype object, filled as they are met


def _code(t, what):
    dtype = t.dtype
    code = _CODE_OF.get(dtype)
    if code is None:
        code = _TENSOR_CODES.get(str(dtype))
        if code is None:
            raise GemmError(GEMM_ERR_UNSUPPORTED_DTYPE, f"{what}: {dtype}")
        _CODE_OF[dtype] = code
    return code


def _elsewhere(t, what, device):
    """The error for a tensor that is not in the memory of GPU `device`: a kernel would follow
    its address all the same.  (A tensor that does not say where it is, without get_device,
    is taken to be there.)"""
    index = t.get_device()
    where = "the host" if index < 0 else f"GPU {index}"
    return GemmError(GEMM_ERR_INVALID_ARG, f"{what}: on {where}, not on GPU {device}")


def _shape(t, what):
    shape = t.shape
    if len(shape) != 2:
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: shape {tuple(shape)}, not a matrix")
    return shape


def _rows(t, shape, what, device, code=None):
    """(address, row stride) of a matrix of that shape whose rows are contiguous, on GPU
    `device` and of type `code` if given; (0, 0) for None."""
    if t is None:
        return 0, 0
    try:
        if t.get_device() != device:
            raise _elsewhere(t, what, device)
    except AttributeError:
        pass
    if t.shape != shape:
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if code is not None and _CODE_OF.get(t.dtype) != code and _code(t, what) != code:
        raise GemmError(GEMM_ERR_UNSUPPORTED_DTYPE, f"{what}: {t.dtype}")
    s0, s1 = t.stride()
    M, N = shape
    if s1 != 1 and N > 1:
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: rows are not contiguous")
    if M == 1 and (s0 & 15 or s0 < N):
        # the stride of a single row says nothing: any sufficient aligned one will do
        s0 = (max(s0, N) + 15) // 16 * 16
    return t.data_ptr(), s0


def _operand(t, R, K, what, device):
    """(address, stride, layout) of an R x K product operand on GPU `device`, either
    dimension contiguous."""
    try:
        if t.get_device() != device:
            raise _elsewhere(t, what, device)
    except AttributeError:
        pass
    s0, s1 = t.stride()
    if s1 == 1 and not (s0 == 1 and R > 1):
        return t.data_ptr(), s0 if R > 1 else (max(s0, K) + 15) // 16 * 16, GEMM_K_MAJOR
    if s0 == 1 or R == 1:
        return t.data_ptr(), s1 if K > 1 else (max(s1, R) + 15) // 16 * 16, GEMM_MN_MAJOR
    raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: neither dimension is contiguous")


def _activation(name):
    try:
        return ACTIVATION_CODES[name]
    except (KeyError, TypeError):
        raise GemmError(GEMM_ERR_INVALID_ARG, f"activation {name!r}") from None


def _vector(t, n, what, device, code=None):
    """Address of a contiguous vector of n elements on GPU `device` (of type `code` if given);
    0 for None."""
    if t is None:
        return 0
    try:
        if t.get_device() != device:
            raise _elsewhere(t, what, device)
    except AttributeError:
        pass
    if t.shape != (n,) or (t.stride() != (1,) and n > 1):
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: not a contiguous vector of {n}")
    if code is not None and _CODE_OF.get(t.dtype) != code and _code(t, what) != code:
        raise GemmError(GEMM_ERR_UNSUPPORTED_DTYPE, f"{what}: {t.dtype}")
    return t.data_ptr()


class Gemm:
    """Owns one library handle on `device`.

    run, run_host: the C entry points' arguments.  rmsnorm, rmsnorm_bwd, linear,
    linear_bwd: the operators around the product on tensors (torch's or any with
    data_ptr, dtype, shape and stride), whose device, types, sizes and row strides the
    calls read off and check; outputs are the caller's tensors too.
    Tensors are used on `stream` (None: the default stream) and must be ready there."""

    def __init__(self, device: int = 0):
        self.handle = gemm_create(device)
        self.device = int(device)
        self._lib = library()

    def close(self):
        if self.handle:
            gemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y, alpha, beta,
            x_factor, dtypes, stream=None):
        return gemm_run(self.handle, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y,
                        alpha, beta, x_factor, dtypes, stream)

    def run_host(self, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D, Y, alpha, beta,
                 x_factor, dtypes, stream=None):
        return gemm_run_host(self.handle, M, N, K, L, A, lda, layoutA, B, ldb, layoutB, C, X, D,
                             Y, alpha, beta, x_factor, dtypes, stream)

    def ring_stats(self, stream=None):
        """Per-CTA ring counters of the last launch (statistics build only):
        a list of GEMM_RING_STAT_WORDS-long lists, CTA by CTA."""
        max_ctas = 1024
        buf = (ctypes.c_uint64 * (max_ctas * GEMM_RING_STAT_WORDS))()
        n = ctypes.c_int(0)
        st = library().gemm_ring_stats(self.handle, _stream(stream), buf, max_ctas,
                                       ctypes.byref(n))
        if st != GEMM_OK:
            raise GemmError(st, "gemm_ring_stats")
        w = GEMM_RING_STAT_WORDS
        return [list(buf[i * w:(i + 1) * w]) for i in range(n.value)]

    def sync_status(self, stream=None):
        return gemm_sync_status(self.handle, stream)

    def set_config(self, cfg=None, **fields):
        if cfg is None and fields:
            cfg = gemm_config_t(**fields)
        gemm_set_config(self.handle, cfg)

    def last_config(self):
        return gemm_last_config(self.handle)

    def rmsnorm(self, x, weight, y, residual=None, h=None, scale=None, rstd=None, eps=1e-6,
                stream=None):
        """y = (x + residual) * rstd * weight; see gemm_rmsnorm in the C header.  An 8-bit
        y (float8_e4m3fn, float8_e5m2) is quantised per row, with its scales in
        `scale`; `h` receives x + residual, `rstd` the rows' factors."""
        shape = _shape(x, "x")
        M, H = shape
        t, dev = _code(x, "x"), self.device
        st = self._lib.gemm_rmsnorm(self.handle, _RMSNORM.pack(
            M, H, t, _code(weight, "weight"), _code(y, "y"), eps, *_rows(x, shape, "x", dev),
            *_rows(residual, shape, "residual", dev, t), _vector(weight, H, "weight", dev),
            *_rows(h, shape, "h", dev, t), *_rows(y, shape, "y", dev),
            _vector(scale, M, "scale", dev, GEMM_F32), _vector(rstd, M, "rstd", dev, GEMM_F32)),
            stream and _stream(stream))
        if st:
            raise GemmError(st, "gemm_rmsnorm")

    def rmsnorm_bwd(self, dy, h, weight, rstd, dx, dweight, dh=None, workspace=None,
                    stream=None):
        """Gradients of x (= of the residual) and of weight; see gemm_rmsnorm_bwd in the C
        header.  `workspace`: a contiguous tensor of at least
        gemm_rmsnorm_bwd_workspace(M, H) bytes."""
        shape = _shape(dy, "dy")
        M, H = shape
        t, dev = _code(dy, "dy"), self.device
        ws, nbytes = None, 0
        if workspace is not None:
            try:
                if workspace.get_device() != dev:
                    raise _elsewhere(workspace, "workspace", dev)
                if not workspace.is_contiguous():    # (its bytes are not where they are counted)
                    raise GemmError(GEMM_ERR_INVALID_ARG, "workspace: not contiguous")
            except AttributeError:
                pass
            ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        st = self._lib.gemm_rmsnorm_bwd(self.handle, _RMSNORM_BWD.pack(
            M, H, t, _code(weight, "weight"), _code(dweight, "dweight"),
            *_rows(dy, shape, "dy", dev), *_rows(h, shape, "h", dev, t),
            _vector(weight, H, "weight", dev), _vector(rstd, M, "rstd", dev, GEMM_F32),
            *_rows(dh, shape, "dh", dev, t), *_rows(dx, shape, "dx", dev, t),
            _vector(dweight, H, "dweight", dev)), ws, nbytes,
            stream and _stream(stream))
        if st:
            raise GemmError(st, "gemm_rmsnorm_bwd")

    def linear(self, a, b, d, bias=None, activation=None, residual=None, z=None, row_scale=None,
               col_scale=None, alpha=1.0, stream=None):
        """d = act(alpha * (a b^T) * row_scale * col_scale + bias) + residual; see gemm_linear
        in the C header.  a [M, K] and b [N, K], either dimension contiguous; activation:
        None, "relu", "gelu", "gelu_tanh" or "silu"; z receives what the activation is applied
        to.  There is no product of full fp32 precision: fp32 a and b are GEMM_TF32's, of whose
        fractions the matrix units read ten bits and drop the rest, up to 2^-10 of each operand
        and always towards zero."""
        M, K = _shape(a, "a")
        N, inner = _shape(b, "b")
        if inner != K:
            raise GemmError(GEMM_ERR_INVALID_ARG, f"b: shape {(N, inner)}, not {(N, K)}")
        dev = self.device
        pa, lda, la = _operand(a, M, K, "a", dev)
        pb, ldb, lb = _operand(b, N, K, "b", dev)
        out = (M, N)
        st = self._lib.gemm_linear(self.handle, _LINEAR.pack(
            M, N, K, _code(a, "a") or GEMM_TF32, _code(b, "b") or GEMM_TF32,
            0 if bias is None else _code(bias, "bias"),
            0 if residual is None else _code(residual, "residual"),
            0 if z is None else _code(z, "z"), _code(d, "d"), la, lb, _activation(activation), alpha,
            pa, lda, pb, ldb, _vector(row_scale, M, "row_scale", dev, GEMM_F32),
            _vector(col_scale, N, "col_scale", dev, GEMM_F32), _vector(bias, N, "bias", dev),
            *_rows(residual, out, "residual", dev), *_rows(z, out, "z", dev),
            *_rows(d, out, "d", dev)),
            stream and _stream(stream))
        if st:
            raise GemmError(st, "gemm_linear")

    def linear_bwd(self, dd, a, b, z=None, activation=None, dz=None, da=None, db=None, dbias=None,
                   accumulate=False, alpha=1.0, stream=None):
        """Gradients of linear from dd, the gradient of d: dz, da, db (added to with
        `accumulate`) and dbias, each where given; see gemm_linear_bwd in the C header.  a is
        read for db only and b for da only: else either may be None."""
        out = _shape(dd, "dd")
        M, N = out
        inner = a if a is not None else b if b is not None else da if da is not None else db
        K = 0 if inner is None else _shape(inner, "a or b")[1]
        t, dev = _code(dd, "dd"), self.device
        rows_a, rows_b = (M, K), (N, K)
        st = self._lib.gemm_linear_bwd(self.handle, _LINEAR_BWD.pack(
            M, N, K, t, 0 if da is None else _code(da, "da"), 0 if db is None else _code(db, "db"),
            0 if dbias is None else _code(dbias, "dbias"), _activation(activation),
            int(accumulate), alpha, *_rows(dd, out, "dd", dev), *_rows(z, out, "z", dev, t),
            *_rows(a, rows_a, "a", dev, t), *_rows(b, rows_b, "b", dev, t),
            *_rows(dz, out, "dz", dev, t), *_rows(da, rows_a, "da", dev),
            *_rows(db, rows_b, "db", dev), _vector(dbias, N, "dbias", dev)),
            stream and _stream(stream))
        if st:
            raise GemmError(st, "gemm_linear_bwd")
