"""ctypes binding of the C ABI in ``include/gemm.h`` (``libdtgemm.so``).

Argument marshalling only: every step of C = A·B runs in the library's CUDA kernels.
The binding never falls back to another implementation -- if the library is missing
or the device is not an sm_103 GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

API_VERSION = 3  # GEMM_API_VERSION the structures below are laid out for
LAYOUT_NN, LAYOUT_TN = 0, 1
DTYPE_F16, DTYPE_BF16, DTYPE_E4M3, DTYPE_E5M2, DTYPE_F32 = 0, 1, 2, 3, 4
LAYOUTS = {"NN": LAYOUT_NN, "TN": LAYOUT_TN}
DTYPES = {"f16": DTYPE_F16, "bf16": DTYPE_BF16, "e4m3": DTYPE_E4M3, "e5m2": DTYPE_E5M2}
KINDS = {"dense": 0, "block_scaled": 1, "sparse24": 2}  # gemm_kind_t
TORCH_TO_DTYPE = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16}
# 8-bit operand types (gemm_run_ex only).
TORCH_TO_DTYPE_EX = {**TORCH_TO_DTYPE, torch.float8_e4m3fn: DTYPE_E4M3, torch.float8_e5m2: DTYPE_E5M2}
# Biases, bias gradients and weight gradients (the linear-layer entry points).
TORCH_TO_DTYPE_F32 = {**TORCH_TO_DTYPE, torch.float32: DTYPE_F32}
OWN_SUMS_BYTES = 4 << 20  # GEMM_OWN_SUMS_BYTES: column sums that need no more use the handle's workspace
ACTS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # gemm_act_t

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ARCH, ERR_CUDA, ERR_TIMEOUT = range(6)
OPT_CONFIG, OPT_TIMEOUT_NS, OPT_MAX_CTAS, OPT_RASTER_GROUP, OPT_FAULT_INJECT, OPT_STREAM_K, \
    OPT_HOST_ROW_CHUNKS, OPT_HOST_COL_CHUNKS, OPT_SK_MIN_BLOCKS, OPT_SPLIT_MIN_BLOCKS, OPT_K_SNAKE = range(11)
CONFIG_AUTO, CONFIG_128x256, CONFIG_128x128, CONFIG_256x256, CONFIG_128x64 = range(5)


class gemm_plan_t(ctypes.Structure):
    _fields_ = [("config", ctypes.c_int32), ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
                ("bk", ctypes.c_int32), ("stages", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64), ("k_blocks", ctypes.c_int64),
                ("grid", ctypes.c_int64), ("threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
                ("dp_tiles", ctypes.c_int64), ("sk_base", ctypes.c_int64), ("sk_extra", ctypes.c_int64),
                ("raster_group", ctypes.c_int64), ("k_snake", ctypes.c_int64)]


class gemm_args_t(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
                ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("c_col_major", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("scale_a", ctypes.c_float), ("scale_b", ctypes.c_float)]


class gemm_linear_args_t(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("Z", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldy", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldz", ctypes.c_int64), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("bias_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("alpha", ctypes.c_float)]


class gemm_dgrad_args_t(ctypes.Structure):
    _fields_ = [("dY", ctypes.c_void_p), ("W", ctypes.c_void_p), ("Z", ctypes.c_void_p), ("dX", ctypes.c_void_p),
                ("dbias", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lddy", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldz", ctypes.c_int64), ("lddx", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("dbias_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta_bias", ctypes.c_float)]


class gemm_wgrad_args_t(ctypes.Structure):
    _fields_ = [("dY", ctypes.c_void_p), ("X", ctypes.c_void_p), ("dW", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lddy", ctypes.c_int64), ("ldx", ctypes.c_int64), ("lddw", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float)]


class gemm_act_grad_args_t(ctypes.Structure):
    _fields_ = [("dY", ctypes.c_void_p), ("Z", ctypes.c_void_p), ("dZ", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64),
                ("lddy", ctypes.c_int64), ("ldz", ctypes.c_int64), ("lddz", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("dbias_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("beta_bias", ctypes.c_float)]


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}" if what else status_string(status))


_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load ``libdtgemm.so``; raises if it has not been built (no silent fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise ImportError(f"{_build.LIB} is missing: build it with dense_tiled_gemm_04_gb300.build.build()")
    lib = ctypes.CDLL(_build.LIB)
    i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "gemm_create": ([ctypes.POINTER(p), ctypes.c_int], i32),
        "gemm_destroy": ([p], i32),
        "gemm_run": ([p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, p], i32),
        "gemm_run_host": ([p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, p], i32),
        "gemm_run_ex": ([p, ctypes.POINTER(gemm_args_t), p], i32),
        "gemm_run_mx": ([p, ctypes.POINTER(gemm_args_t), p, p, p], i32),
        "gemm_mx_scale_bytes": ([i64, i64], i64),
        "gemm_run_sp": ([p, ctypes.POINTER(gemm_args_t), p, p], i32),
        "gemm_sp_meta_bytes": ([i64, i64], i64),
        "gemm_sp_compress": ([p, p, i64, i64, i64, i32, p, i64, p, p, p], i32),
        "gemm_mx_pack_scales": ([p, p, i64, i64, i64, p, p], i32),
        "gemm_sync_status": ([p, p], i32),
        "gemm_error_info": ([p, ctypes.POINTER(i32)], i32),
        "gemm_set_option": ([p, i32, i64], i32),
        "gemm_get_option": ([p, i32, ctypes.POINTER(i64)], i32),
        "gemm_query_plan": ([p, i64, i64, i64, i32, i32, ctypes.POINTER(gemm_plan_t)], i32),
        "gemm_query_plan_kind": ([p, i64, i64, i64, i32, i32, i32, ctypes.POINTER(gemm_plan_t)], i32),
        "gemm_check_args": ([p, p, p, i64, i64, i64, i64, i64, i64, i32, i32], i32),
        "gemm_tile_coord": ([i64, i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)], i32),
        "gemm_run_noalloc": ([p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, p, ctypes.POINTER(i32)], i32),
        "gemm_run_linear": ([p, ctypes.POINTER(gemm_linear_args_t), p], i32),
        "gemm_run_linear_dgrad": ([p, ctypes.POINTER(gemm_dgrad_args_t), p], i32),
        "gemm_run_linear_wgrad": ([p, ctypes.POINTER(gemm_wgrad_args_t), p], i32),
        "gemm_run_act_grad": ([p, ctypes.POINTER(gemm_act_grad_args_t), p], i32),
        "gemm_bias_grad_workspace_bytes": ([i64, i64], i64),
        "gemm_status_string": ([i32], ctypes.c_char_p),
        "gemm_api_version": ([], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if lib.gemm_api_version() != API_VERSION:
        raise ImportError(f"{_build.LIB} implements API version {lib.gemm_api_version()}, this binding "
                          f"version {API_VERSION}: rebuild it with dense_tiled_gemm_04_gb300.build.build()")
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().gemm_status_string(int(status)).decode()


def check_args(A: int, B: int, C: int, M, N, K, lda, ldb, ldc, layout: int, dtype: int) -> int:
    """gemm_check_args on raw addresses (no GPU needed)."""
    return int(load().gemm_check_args(A or None, B or None, C or None, M, N, K, lda, ldb, ldc, layout, dtype))


def mx_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the chunked block-scale layout for `rows` rows and K elements of K."""
    return int(load().gemm_mx_scale_bytes(rows, K))


def sp_meta_bytes(M: int, K: int) -> int:
    """Bytes of the chunked 2:4 sparsity metadata for M rows and K."""
    return int(load().gemm_sp_meta_bytes(M, K))


def bias_grad_workspace_bytes(M: int, cols: int) -> int:
    """Bytes of workspace for the column sums of an M x cols matrix."""
    return int(load().gemm_bias_grad_workspace_bytes(M, cols))


def _sums_bytes(M: int, cols: int) -> int:
    """bias_grad_workspace_bytes without a call into the library, which a small call would notice."""
    return 4 * -(-M // 32) * (-(-cols // 64) * 64)


def tile_coord(tile: int, tiles_m: int, tiles_n: int, group_m: int):
    tm, tn = ctypes.c_int64(), ctypes.c_int64()
    st = load().gemm_tile_coord(tile, tiles_m, tiles_n, group_m, ctypes.byref(tm), ctypes.byref(tn))
    if st != OK:
        raise GemmError(st, "gemm_tile_coord")
    return tm.value, tn.value


def _ld(t: torch.Tensor) -> int:
    """Leading dimension of a 2-D row-major tensor (one-row tensors: the padded row length)."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError("expected unit stride along the last dimension (row-major)")
    if t.size(0) <= 1:
        align = 16 // t.element_size()  # a TMA row pitch is a multiple of 16 bytes
        return max(-(-t.size(1) // align) * align, align)
    return t.stride(0)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def empty_output(M: int, N: int, dtype: torch.dtype, device) -> torch.Tensor:
    """An M x N output whose row pitch is a multiple of 8 elements (TMA alignment)."""
    ldc = max(-(-N // 8) * 8, 8)
    return torch.empty((M, ldc), dtype=dtype, device=device)[:, :N]


# The checks of the linear-layer calls run for every call, also those of a few microseconds: they
# touch each tensor's attributes as few times as they can.
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream(device).cuda_stream, without the wrapper


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _matrix(t: torch.Tensor, what: str, rows: int, cols: int, dtype: torch.dtype, device: int) -> int:
    """Check a 2-D tensor argument and return its leading dimension (one-row tensors: the padded row length)."""
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must have shape {(rows, cols)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what} must be on cuda:{device}, not {t.device}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride along the last dimension (row-major)")
    if rows <= 1:
        align = 16 // t.element_size()
        return max(-(-cols // align) * align, align)
    return ld


def _vector(t: torch.Tensor, what: str, n: int, dtype: torch.dtype, device: int) -> int:
    """Check a dense 1-D tensor argument, float32 or `dtype`, and return its element type's code."""
    if t.dtype is not torch.float32 and t.dtype is not dtype:
        raise TypeError(f"{what} must be float32 or {dtype}, not {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride() != (1,)):
        raise ValueError(f"{what} must be a dense vector of {n} elements")
    if t.get_device() != device:
        raise ValueError(f"{what} must be on cuda:{device}, not {t.device}")
    return TORCH_TO_DTYPE_F32[t.dtype]


def _act(name) -> int:
    if name not in ACTS:
        raise ValueError(f"unknown activation {name!r}: one of {sorted(k for k in ACTS if k)}")
    return ACTS[name]


def _new(rows: int, cols: int, dtype: torch.dtype, device: int, stream) -> torch.Tensor:
    """A new output that belongs to `stream` (None: the current stream), so that its memory is not
    handed out again while the stream still uses it."""
    if stream is None:
        return _padded_output(rows, cols, dtype, device)
    if not hasattr(stream, "cuda_stream"):
        # (ExternalStream(0) would be a stream of the pool.)
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return _padded_output(rows, cols, dtype, device)


def _padded_output(rows: int, cols: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A rows x cols output whose row pitch is a multiple of 16 bytes."""
    align = 4 if dtype is torch.float32 else 8
    ld = max(-(-cols // align) * align, align)
    t = torch.empty((rows, ld), dtype=dtype, device=device)
    return t if ld == cols else t[:, :cols]


class Gemm:
    """A library handle bound to one CUDA device.

    Its calls share a workspace: make them from one host thread at a time, on one stream or on streams that are ordered.
    A captured graph uses it too: keep the handle open, and its other calls ordered with the replays."""

    def __init__(self, device=None):
        lib = load()
        if device is None:
            device = torch.cuda.current_device()
        self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        self._index = self.device.index or 0
        h = ctypes.c_void_p()
        st = lib.gemm_create(ctypes.byref(h), self.device.index or 0)
        if st != OK:
            raise GemmError(st, "gemm_create")
        self._h = h
        self._lib = lib

    # -------------------------------------------------------------- lifecycle
    def close(self):
        if getattr(self, "_h", None):
            st = self._lib.gemm_destroy(self._h)
            self._h = None
            if st != OK:
                raise GemmError(st, "gemm_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # -------------------------------------------------------------- options
    def set_option(self, opt: int, value: int):
        st = self._lib.gemm_set_option(self._h, opt, int(value))
        if st != OK:
            raise GemmError(st, "gemm_set_option")

    def get_option(self, opt: int) -> int:
        v = ctypes.c_int64()
        st = self._lib.gemm_get_option(self._h, opt, ctypes.byref(v))
        if st != OK:
            raise GemmError(st, "gemm_get_option")
        return v.value

    def plan(self, M, N, K, layout="NN", dtype="f16", kind: str = "dense") -> dict:
        """The launch the entry point for `kind` ("dense", "block_scaled", "sparse24") would make."""
        pl = gemm_plan_t()
        st = self._lib.gemm_query_plan_kind(self._h, M, N, K, LAYOUTS[layout], DTYPES[dtype], KINDS[kind],
                                            ctypes.byref(pl))
        if st != OK:
            raise GemmError(st, "gemm_query_plan_kind")
        return {f: getattr(pl, f) for f, _ in gemm_plan_t._fields_}

    def error_info(self):
        arr = (ctypes.c_int32 * 4)()
        self._lib.gemm_error_info(self._h, arr)
        return list(arr)

    # -------------------------------------------------------------- compute
    def run_raw(self, A: int, B: int, C: int, M, N, K, lda, ldb, ldc, layout: int, dtype: int, stream: int) -> int:
        """gemm_run on raw device addresses; returns the status code."""
        return int(self._lib.gemm_run(self._h, A or None, B or None, C or None, M, N, K, lda, ldb, ldc,
                                      layout, dtype, stream or None))

    def run(self, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, layout: str = "NN",
            stream=None) -> torch.Tensor:
        """C = A·B (NN: B is K x N) or A·B^T (TN: B is N x K) on device tensors; async on `stream`."""
        M, K = A.shape
        N = B.shape[1] if layout == "NN" else B.shape[0]
        if (B.shape[0] if layout == "NN" else B.shape[1]) != K:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, layout {layout}")
        if A.dtype != B.dtype or A.dtype not in TORCH_TO_DTYPE:
            raise TypeError("A and B must both be float16 or both bfloat16")
        if C is None:
            C = empty_output(M, N, A.dtype, A.device)
        if C.shape != (M, N) or C.dtype != A.dtype:
            raise ValueError("C has the wrong shape or dtype")
        st = self.run_raw(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, _ld(A), _ld(B), _ld(C),
                          LAYOUTS[layout], TORCH_TO_DTYPE[A.dtype], _stream_ptr(stream))
        if st != OK:
            raise GemmError(st, "gemm_run")
        return C

    def run_ex_raw(self, A: int, B: int, C: int, M, N, K, lda, ldb, ldc, layout: int, dtype: int, alpha: float,
                   beta: float, c_col_major: int, stream: int, out_dtype: int | None = None, scale_a: float = 1.0,
                   scale_b: float = 1.0) -> int:
        """gemm_run_ex on raw device addresses:
        C = alpha * scale_a * scale_b * A·B + beta * C (row- or column-major C)."""
        a = gemm_args_t(A or None, B or None, C or None, M, N, K, lda, ldb, ldc, layout, dtype, alpha, beta,
                        c_col_major, dtype if out_dtype is None else out_dtype, scale_a, scale_b)
        return int(self._lib.gemm_run_ex(self._h, ctypes.byref(a), stream or None))

    def run_ex(self, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, layout: str = "NN",
               out_dtype: torch.dtype | None = None, alpha: float = 1.0, beta: float = 0.0, scale_a: float = 1.0,
               scale_b: float = 1.0, c_col_major: bool = False, stream=None) -> torch.Tensor:
        """C = alpha * scale_a * scale_b * A·B + beta * C on device tensors; A, B 16-bit or 8-bit
        (float8_e4m3fn / float8_e5m2), C float16 or bfloat16.  With c_col_major, ``C`` is the
        N x M row-major tensor holding C transposed.  Async on `stream`."""
        M, K = A.shape
        N = B.shape[1] if layout == "NN" else B.shape[0]
        if (B.shape[0] if layout == "NN" else B.shape[1]) != K:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, layout {layout}")
        if A.dtype != B.dtype or A.dtype not in TORCH_TO_DTYPE_EX:
            raise TypeError("A and B must have the same 16-bit or 8-bit float type")
        if out_dtype is None:
            out_dtype = C.dtype if C is not None else (A.dtype if A.dtype in TORCH_TO_DTYPE else torch.bfloat16)
        if out_dtype not in TORCH_TO_DTYPE:
            raise TypeError("C must be float16 or bfloat16")
        shape = (N, M) if c_col_major else (M, N)
        if C is None:
            C = empty_output(*shape, out_dtype, A.device)
        if tuple(C.shape) != shape or C.dtype != out_dtype:
            raise ValueError("C has the wrong shape or dtype")
        st = self.run_ex_raw(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, _ld(A), _ld(B), _ld(C),
                             LAYOUTS[layout], TORCH_TO_DTYPE_EX[A.dtype], alpha, beta, int(c_col_major),
                             _stream_ptr(stream), TORCH_TO_DTYPE[out_dtype], scale_a, scale_b)
        if st != OK:
            raise GemmError(st, "gemm_run_ex")
        return C

    def pack_scales(self, sf: torch.Tensor, K: int | None = None, stream=None) -> torch.Tensor:
        """Row-major E8M0 exponents (rows x ceil(K/32), uint8, on the device) -> the chunked
        layout gemm_run_mx reads, in a new uint8 tensor (gemm_mx_pack_scales, async)."""
        if sf.dtype != torch.uint8 or sf.dim() != 2 or (sf.size(1) > 1 and sf.stride(1) != 1):
            raise ValueError("expected a 2-D row-major uint8 tensor")
        rows, kblocks = sf.shape
        K = 32 * kblocks if K is None else K
        if -(-K // 32) != kblocks:
            raise ValueError(f"{kblocks} K blocks do not cover K = {K}")
        out = torch.empty(max(mx_scale_bytes(rows, K), 16), dtype=torch.uint8, device=sf.device)
        ld = sf.stride(0) if rows > 1 else max(kblocks, 1)
        st = self._lib.gemm_mx_pack_scales(self._h, sf.data_ptr() or None, rows, kblocks, ld, out.data_ptr(),
                                           _stream_ptr(stream))
        if st != OK:
            raise GemmError(st, "gemm_mx_pack_scales")
        return out

    def run_mx_raw(self, A: int, B: int, C: int, sfa: int, sfb: int, M, N, K, lda, ldb, ldc, layout: int, dtype: int,
                   out_dtype: int, alpha: float = 1.0, beta: float = 0.0, c_col_major: int = 0, scale_a: float = 1.0,
                   scale_b: float = 1.0, stream: int = 0) -> int:
        """gemm_run_mx on raw device addresses; returns the status code."""
        a = gemm_args_t(A or None, B or None, C or None, M, N, K, lda, ldb, ldc, layout, dtype, alpha, beta,
                        c_col_major, out_dtype, scale_a, scale_b)
        return int(self._lib.gemm_run_mx(self._h, ctypes.byref(a), sfa or None, sfb or None, stream or None))

    def run_mx(self, A: torch.Tensor, B: torch.Tensor, sfa: torch.Tensor, sfb: torch.Tensor,
               C: torch.Tensor | None = None, layout: str = "NN", out_dtype: torch.dtype = torch.bfloat16,
               alpha: float = 1.0, beta: float = 0.0, scale_a: float = 1.0, scale_b: float = 1.0,
               c_col_major: bool = False, stream=None) -> torch.Tensor:
        """C = alpha * scale_a * scale_b * (A·B with per-tile E8M0 scales) + beta * C on device
        tensors: A, B float8_e4m3fn / float8_e5m2; sfa, sfb the chunked scales (pack_scales).
        Async on `stream`."""
        M, K = A.shape
        N = B.shape[1] if layout == "NN" else B.shape[0]
        if (B.shape[0] if layout == "NN" else B.shape[1]) != K:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, layout {layout}")
        if A.dtype != B.dtype or A.dtype not in (torch.float8_e4m3fn, torch.float8_e5m2):
            raise TypeError("A and B must have the same 8-bit float type")
        if out_dtype not in TORCH_TO_DTYPE:
            raise TypeError("C must be float16 or bfloat16")
        for t, rows, what in ((sfa, M, "sfa"), (sfb, N, "sfb")):
            if t.dtype != torch.uint8 or t.numel() < mx_scale_bytes(rows, K):
                raise ValueError(f"{what} must hold {mx_scale_bytes(rows, K)} bytes of packed scales")
        shape = (N, M) if c_col_major else (M, N)
        if C is None:
            C = empty_output(*shape, out_dtype, A.device)
        if tuple(C.shape) != shape or C.dtype != out_dtype:
            raise ValueError("C has the wrong shape or dtype")
        st = self.run_mx_raw(A.data_ptr(), B.data_ptr(), C.data_ptr(), sfa.data_ptr(), sfb.data_ptr(), M, N, K, _ld(A),
                             _ld(B), _ld(C), LAYOUTS[layout], TORCH_TO_DTYPE_EX[A.dtype], TORCH_TO_DTYPE[out_dtype],
                             alpha, beta, int(c_col_major), scale_a, scale_b, _stream_ptr(stream))
        if st != OK:
            raise GemmError(st, "gemm_run_mx")
        return C

    def sp_compress(self, A: torch.Tensor, stream=None):
        """2:4 compression of a dense fp16/bf16 device matrix (gemm_sp_compress, async):
        returns (Ac: M x K/2 kept values, meta: chunked metadata bytes, bad: 1-element int32
        device tensor counting groups with more than two non-zeros)."""
        if A.dtype not in TORCH_TO_DTYPE or A.dim() != 2:
            raise TypeError("A must be a 2-D float16 or bfloat16 tensor")
        M, K = A.shape
        if K % 4:
            raise ValueError("K must be a multiple of 4")
        Ac = empty_output(M, K // 2, A.dtype, A.device)
        meta = torch.empty(max(sp_meta_bytes(M, K), 16), dtype=torch.uint8, device=A.device)
        bad = torch.zeros(1, dtype=torch.int32, device=A.device)
        st = self._lib.gemm_sp_compress(self._h, A.data_ptr() or None, M, K, _ld(A), TORCH_TO_DTYPE[A.dtype],
                                        Ac.data_ptr() or None, _ld(Ac), meta.data_ptr(), bad.data_ptr(),
                                        _stream_ptr(stream))
        if st != OK:
            raise GemmError(st, "gemm_sp_compress")
        return Ac, meta, bad

    def run_sp_raw(self, Ac: int, B: int, C: int, meta: int, M, N, K, lda, ldb, ldc, layout: int, dtype: int,
                   alpha: float = 1.0, beta: float = 0.0, c_col_major: int = 0, stream: int = 0) -> int:
        """gemm_run_sp on raw device addresses (Ac: the compressed A, lda its pitch; K logical)."""
        a = gemm_args_t(Ac or None, B or None, C or None, M, N, K, lda, ldb, ldc, layout, dtype, alpha, beta,
                        c_col_major, dtype, 1.0, 1.0)
        return int(self._lib.gemm_run_sp(self._h, ctypes.byref(a), meta or None, stream or None))

    def run_sp(self, Ac: torch.Tensor, B: torch.Tensor, meta: torch.Tensor, C: torch.Tensor | None = None,
               layout: str = "NN", alpha: float = 1.0, beta: float = 0.0, c_col_major: bool = False,
               stream=None) -> torch.Tensor:
        """C = alpha * A·B + beta * C with A 2:4-sparse, given as (Ac, meta) from sp_compress.
        K = 2 * Ac's columns.  Async on `stream`."""
        M, K = Ac.shape[0], 2 * Ac.shape[1]
        N = B.shape[1] if layout == "NN" else B.shape[0]
        if (B.shape[0] if layout == "NN" else B.shape[1]) != K:
            raise ValueError(f"shape mismatch: Ac {tuple(Ac.shape)}, B {tuple(B.shape)}, layout {layout}")
        if Ac.dtype != B.dtype or Ac.dtype not in TORCH_TO_DTYPE:
            raise TypeError("Ac and B must both be float16 or both bfloat16")
        if meta.dtype != torch.uint8 or meta.numel() < sp_meta_bytes(M, K):
            raise ValueError(f"meta must hold {sp_meta_bytes(M, K)} bytes")
        shape = (N, M) if c_col_major else (M, N)
        if C is None:
            C = empty_output(*shape, Ac.dtype, Ac.device)
        if tuple(C.shape) != shape or C.dtype != Ac.dtype:
            raise ValueError("C has the wrong shape or dtype")
        st = self.run_sp_raw(Ac.data_ptr(), B.data_ptr(), C.data_ptr(), meta.data_ptr(), M, N, K, _ld(Ac), _ld(B),
                             _ld(C), LAYOUTS[layout], TORCH_TO_DTYPE[Ac.dtype], alpha, beta, int(c_col_major),
                             _stream_ptr(stream))
        if st != OK:
            raise GemmError(st, "gemm_run_sp")
        return C

    def run_host(self, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, layout: str = "NN", stream=None) -> int:
        """gemm_run_host on CPU tensors (pin them for DMA copies); synchronous; returns the status."""
        M, K = A.shape
        N = C.shape[1]
        return int(self._lib.gemm_run_host(self._h, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                           _ld(A), _ld(B), _ld(C), LAYOUTS[layout], TORCH_TO_DTYPE[A.dtype],
                                           _stream_ptr(stream) or None))

    # -------------------------------------------------------------- linear layers
    # (_ptr: the stream's address, where the caller has looked it up)
    def linear(self, X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str | None = None,
               residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
               preact: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, alpha: float = 1.0,
               stream=None, _ptr=None) -> torch.Tensor:
        """Y = act(alpha * X·W^T + bias) + residual (gemm_run_linear): X (M x K) and W (N x K) 16-bit or
        8-bit floats, Y, residual and preact float16 or bfloat16, bias float32 or Y's type.  ``preact``, if
        given, receives alpha * X·W^T + bias; ``out`` may be ``residual`` itself.  Async on `stream`."""
        dt, dev = X.dtype, self._index
        in_code = TORCH_TO_DTYPE_EX.get(dt)
        if in_code is None:
            raise TypeError("X and W must have the same 16-bit or 8-bit float type")
        if X.dim() != 2 or W.dim() != 2:
            raise ValueError("expected 2-D tensors")
        (M, K), N = X.shape, W.shape[0]
        if out_dtype is None:
            out_dtype = out.dtype if out is not None else (dt if in_code <= DTYPE_BF16 else torch.bfloat16)
        out_code = TORCH_TO_DTYPE.get(out_dtype)
        if out_code is None or (in_code <= DTYPE_BF16 and out_code != in_code):
            raise TypeError("Y must be float16 or bfloat16, and of the operands' type if that is 16-bit")
        ldx, ldw = _matrix(X, "X", M, K, dt, dev), _matrix(W, "W", N, K, dt, dev)
        bias_p = res_p = z_p = bias_code = ldr = ldz = 0
        if bias is not None:
            bias_code, bias_p = _vector(bias, "bias", N, out_dtype, dev), bias.data_ptr()
        if residual is not None:
            ldr, res_p = _matrix(residual, "residual", M, N, out_dtype, dev), residual.data_ptr()
        if preact is not None:
            ldz, z_p = _matrix(preact, "preact", M, N, out_dtype, dev), preact.data_ptr()
        if out is None:
            out = _new(M, N, out_dtype, dev, stream)
        ldy = _matrix(out, "out", M, N, out_dtype, dev)
        a = gemm_linear_args_t(X.data_ptr(), W.data_ptr(), out.data_ptr(), bias_p, res_p, z_p, M, N, K, ldx, ldw, ldy, ldr,
                               ldz, in_code, out_code, bias_code, _act(act), alpha)
        st = self._lib.gemm_run_linear(self._h, ctypes.byref(a), _stream_of(stream, dev) if _ptr is None else _ptr)
        if st != OK:
            raise GemmError(st, "gemm_run_linear")
        return out

    def linear_dgrad(self, dY: torch.Tensor, W: torch.Tensor, Z: torch.Tensor | None = None, act: str | None = None,
                     out: torch.Tensor | None = None, dbias: torch.Tensor | None = None, alpha: float = 1.0,
                     beta_bias: float = 0.0, stream=None, _ptr=None) -> torch.Tensor:
        """dX = (alpha * dY·W) * act'(Z) (gemm_run_linear_dgrad): dY (M x N), W (N x K), Z (M x K, what the
        layer below kept; not read without an activation) of one 16-bit type.  ``dbias`` (K, float32 or that type), if given, becomes
        beta_bias * dbias + the column sums of dX.  Async on `stream`."""
        dt, dev, code = dY.dtype, self._index, _act(act)
        dt_code = TORCH_TO_DTYPE.get(dt)
        if dt_code is None:
            raise TypeError("dY and W must both be float16 or both bfloat16")
        if dY.dim() != 2 or W.dim() != 2:
            raise ValueError("expected 2-D tensors")
        (M, N), K = dY.shape, W.shape[1]
        if code == 0:
            Z = None  # not read
        elif Z is None:
            raise ValueError("act needs its pre-activation Z")
        lddy, ldw = _matrix(dY, "dY", M, N, dt, dev), _matrix(W, "W", N, K, dt, dev)
        z_p = db_p = ldz = db_code = ws_p = ws_bytes = 0
        if Z is not None:
            ldz, z_p = _matrix(Z, "Z", M, K, dt, dev), Z.data_ptr()
        if out is None:
            out = _new(M, K, dt, dev, stream)
        lddx = _matrix(out, "out", M, K, dt, dev)
        if dbias is not None:
            db_code, db_p = _vector(dbias, "dbias", K, dt, dev), dbias.data_ptr()
            ws_bytes = _sums_bytes(M, K)
            if ws_bytes > OWN_SUMS_BYTES:
                ws = _new(1, ws_bytes // 4, torch.float32, dev, stream)
                ws_p = ws.data_ptr()
        a = gemm_dgrad_args_t(dY.data_ptr(), W.data_ptr(), z_p, out.data_ptr(), db_p, ws_p, ws_bytes, M, N, K, lddy, ldw,
                              ldz, lddx, dt_code, db_code, code, alpha, beta_bias)
        st = self._lib.gemm_run_linear_dgrad(self._h, ctypes.byref(a), _stream_of(stream, dev) if _ptr is None else _ptr)
        if st != OK:
            raise GemmError(st, "gemm_run_linear_dgrad")
        return out

    def linear_wgrad(self, dY: torch.Tensor, X: torch.Tensor, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype | None = None, alpha: float = 1.0, beta: float = 0.0,
                     stream=None, _ptr=None) -> torch.Tensor:
        """dW = alpha * dY^T·X + beta * dW (gemm_run_linear_wgrad): dY (M x N) and X (M x K) of one 16-bit
        type, dW (N x K) float32 (the default) or that type.  Async on `stream`."""
        dt, dev = dY.dtype, self._index
        dt_code = TORCH_TO_DTYPE.get(dt)
        if dt_code is None:
            raise TypeError("dY and X must both be float16 or both bfloat16")
        if dY.dim() != 2 or X.dim() != 2:
            raise ValueError("expected 2-D tensors")
        if out is None and beta != 0.0:
            raise ValueError("beta adds to an existing dW: pass it as out")
        (M, N), K = dY.shape, X.shape[1]
        if out_dtype is None:
            out_dtype = out.dtype if out is not None else torch.float32
        if out_dtype is not torch.float32 and out_dtype is not dt:
            raise TypeError("dW must be float32 or of the operands' type")
        lddy, ldx = _matrix(dY, "dY", M, N, dt, dev), _matrix(X, "X", M, K, dt, dev)
        if out is None:
            out = _new(N, K, out_dtype, dev, stream)
        lddw = _matrix(out, "out", N, K, out_dtype, dev)
        a = gemm_wgrad_args_t(dY.data_ptr(), X.data_ptr(), out.data_ptr(), M, N, K, lddy, ldx, lddw, dt_code,
                              TORCH_TO_DTYPE_F32[out_dtype], alpha, beta)
        st = self._lib.gemm_run_linear_wgrad(self._h, ctypes.byref(a), _stream_of(stream, dev) if _ptr is None else _ptr)
        if st != OK:
            raise GemmError(st, "gemm_run_linear_wgrad")
        return out

    def act_grad(self, dY: torch.Tensor, Z: torch.Tensor | None = None, act: str | None = None,
                 out: torch.Tensor | None = None, dbias: torch.Tensor | None = None, beta_bias: float = 0.0,
                 sums_only: bool = False, stream=None, _ptr=None) -> torch.Tensor | None:
        """dZ = dY * act'(Z) (gemm_run_act_grad): dY and Z (M x N; not read without an activation) of one 16-bit
        type; ``out`` may be dY itself.  ``dbias`` as for linear_dgrad, with N columns.  With ``sums_only`` dZ is not written (and None is
        returned).  Async on `stream`."""
        dt, dev, code = dY.dtype, self._index, _act(act)
        dt_code = TORCH_TO_DTYPE.get(dt)
        if dt_code is None or dY.dim() != 2:
            raise TypeError("dY must be a 2-D float16 or bfloat16 tensor")
        M, N = dY.shape
        if code == 0:
            Z = None  # not read
        elif Z is None:
            raise ValueError("act needs its pre-activation Z")
        if sums_only and (out is not None or dbias is None):
            raise ValueError("sums_only writes dbias and no dZ")
        lddy = _matrix(dY, "dY", M, N, dt, dev)
        z_p = dz_p = db_p = ldz = lddz = db_code = ws_p = ws_bytes = 0
        if Z is not None:
            ldz, z_p = _matrix(Z, "Z", M, N, dt, dev), Z.data_ptr()
        if not sums_only:
            if out is None:
                out = _new(M, N, dt, dev, stream)
            lddz, dz_p = _matrix(out, "out", M, N, dt, dev), out.data_ptr()
        if dbias is not None:
            db_code, db_p = _vector(dbias, "dbias", N, dt, dev), dbias.data_ptr()
            ws_bytes = _sums_bytes(M, N)
            if ws_bytes > OWN_SUMS_BYTES:
                ws = _new(1, ws_bytes // 4, torch.float32, dev, stream)
                ws_p = ws.data_ptr()
        a = gemm_act_grad_args_t(dY.data_ptr(), z_p, dz_p, db_p, ws_p, ws_bytes, M, N, lddy, ldz, lddz, dt_code, db_code,
                                 code, beta_bias)
        st = self._lib.gemm_run_act_grad(self._h, ctypes.byref(a), _stream_of(stream, dev) if _ptr is None else _ptr)
        if st != OK:
            raise GemmError(st, "gemm_run_act_grad")
        return out

    def sync_status(self, stream=None) -> int:
        return int(self._lib.gemm_sync_status(self._h, _stream_ptr(stream) or None))


# The handles of the module functions, one per (device, stream): a handle's workspace (stream-K parts and counters, column
# sums) serves one call at a time, so calls on streams that are not ordered need one each, and a captured graph keeps
# that of the stream it was captured on.  A call may be two launches: the lock keeps those of two host threads apart.
_default: dict = {}
_default_lock = threading.Lock()


def _default_handle(device: int, stream: int):
    """The (handle, lock) of a device's stream."""
    h = _default.get((device, stream))
    if h is None:
        with _default_lock:
            h = _default.get((device, stream))
            if h is None:
                h = _default[device, stream] = (Gemm(device), threading.RLock())
    return h


def _default_of(t: torch.Tensor, stream):
    """The (handle, lock) of a tensor's device and a stream, and the stream's address."""
    device = t.get_device()
    if device < 0:
        raise ValueError("expected CUDA tensors")
    ptr = _raw_stream(device) if stream is None else _stream_of(stream, device)
    h, lock = _default.get((device, ptr)) or _default_handle(device, ptr)
    return h, lock, ptr


def matmul(A: torch.Tensor, B: torch.Tensor, layout: str = "NN", out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """C = A·B with the library's kernel, on a default handle of the stream (so calls on several streams and from
    several threads do not disturb one another).  A captured graph keeps that of its capture stream: replays of
    graphs captured on one stream must not overlap."""
    dev = A.device.index if A.device.index is not None else torch.cuda.current_device()
    h, lock = _default_handle(dev, _stream_ptr(stream))
    with lock:
        return h.run(A, B, out, layout, stream)


def linear(X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str | None = None,
           residual: torch.Tensor | None = None, out: torch.Tensor | None = None, preact: torch.Tensor | None = None,
           out_dtype: torch.dtype | None = None, alpha: float = 1.0, stream=None) -> torch.Tensor:
    """Gemm.linear on a default handle of the stream (see matmul)."""
    h, lock, ptr = _default_of(X, stream)
    with lock:
        return h.linear(X, W, bias, act, residual, out, preact, out_dtype, alpha, stream, ptr)


def linear_dgrad(dY: torch.Tensor, W: torch.Tensor, Z: torch.Tensor | None = None, act: str | None = None,
                 out: torch.Tensor | None = None, dbias: torch.Tensor | None = None, alpha: float = 1.0,
                 beta_bias: float = 0.0, stream=None) -> torch.Tensor:
    """Gemm.linear_dgrad on a default handle of the stream (see matmul)."""
    h, lock, ptr = _default_of(dY, stream)
    with lock:
        return h.linear_dgrad(dY, W, Z, act, out, dbias, alpha, beta_bias, stream, ptr)


def linear_wgrad(dY: torch.Tensor, X: torch.Tensor, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None, alpha: float = 1.0, beta: float = 0.0, stream=None) -> torch.Tensor:
    """Gemm.linear_wgrad on a default handle of the stream (see matmul)."""
    h, lock, ptr = _default_of(dY, stream)
    with lock:
        return h.linear_wgrad(dY, X, out, out_dtype, alpha, beta, stream, ptr)


def act_grad(dY: torch.Tensor, Z: torch.Tensor | None = None, act: str | None = None, out: torch.Tensor | None = None,
             dbias: torch.Tensor | None = None, beta_bias: float = 0.0, sums_only: bool = False,
             stream=None) -> torch.Tensor | None:
    """Gemm.act_grad on a default handle of the stream (see matmul)."""
    h, lock, ptr = _default_of(dY, stream)
    with lock:
        return h.act_grad(dY, Z, act, out, dbias, beta_bias, sums_only, stream, ptr)
