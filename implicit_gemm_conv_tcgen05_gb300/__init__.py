"""Python binding of libigc.so, the GB300 (sm_103a) tensor-core GEMM and
implicit-GEMM convolution library.

The functions here have the names of the C ABI (include/igc.h) and do
argument marshalling only: they take torch tensors (device memory) and the
current torch CUDA stream, pass raw pointers, sizes and strides to the C
entry points, and raise IGCError on a non-zero status.  All computation runs
in the library's CUDA kernels; there is no CPU fallback.  If the library is
missing and cannot be built, importing the binding's functions raises.
"""

from __future__ import annotations

import array
import ctypes
import os
import re
import threading
import weakref

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
HEADER = os.path.join(_ROOT, "include", "igc.h")
DEBUG_HEADER = os.path.join(_ROOT, "include", "igc_debug.h")
FFN_HEADER = os.path.join(_ROOT, "include", "igc_ffn.h")
LAYERS_HEADER = os.path.join(_ROOT, "include", "igc_layers.h")

IGC_OK = 0
IGC_ERR_INVALID_ARG = 1
IGC_ERR_MISALIGNED = 2
IGC_ERR_UNSUPPORTED = 3
IGC_ERR_CUDA = 4
IGC_ERR_DEVICE_TIMEOUT = 5
IGC_ERR_WORKSPACE = 6
IGC_F32 = 0
IGC_F16 = 1
IGC_BF16 = 2
IGC_ACT_NONE = 0
IGC_ACT_RELU = 1
IGC_ACT_GELU = 2
IGC_ACT_GELU_TANH = 3
IGC_ACT_SILU = 4

_lock = threading.Lock()
_lib = None


class IGCError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def library_path() -> str:
    from . import build as _b
    return _b.LIB


def lib() -> ctypes.CDLL:
    """The loaded libigc.so (built in-tree on first use if out of date)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            from . import build as _b
            path = _b.build()
            if not os.path.exists(path):
                raise ImportError(f"libigc.so missing at {path}")
            L = ctypes.CDLL(path)
            i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
            L.gemm_f16.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp]
            L.gemm_f16.restype = i32
            L.gemm_bf16.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp]
            L.gemm_bf16.restype = i32
            L.gemm_s8_zp.argtypes = [i64, i64, i64, vp, i32, i64, vp, i32, i64,
                                     ctypes.c_int32, vp, ctypes.c_int32, vp,
                                     vp, i64, vp, i64, ctypes.c_float, vp, vp, sz, vp]
            L.gemm_s8_zp.restype = i32
            L.gemm_s8_zp_prepare.argtypes = [i64, i64, i64, vp, i32, i64, vp, i32, i64, vp, sz, vp]
            L.gemm_s8_zp_prepare.restype = i32
            L.gemm_s8_zp_run.argtypes = [i64, i64, i64, i32, i32, ctypes.c_int32, vp,
                                         ctypes.c_int32, vp, vp, i64, vp, i64, ctypes.c_float,
                                         vp, vp, sz, vp]
            L.gemm_s8_zp_run.restype = i32
            L.gemm_s8_zp_dequant.argtypes = [i64, i64, i64, vp, i32, i64, vp, i32, i64,
                                             ctypes.c_int32, vp, ctypes.c_int32, vp,
                                             vp, vp, vp, vp, i64, vp, sz, vp]
            L.gemm_s8_zp_dequant.restype = i32
            L.gemm_s8_zp_noalloc.argtypes = [i64, i64, i64, vp, i32, i64, vp, i32, i64,
                                             ctypes.c_int32, vp, ctypes.c_int32, vp,
                                             vp, i64, vp, i64, ctypes.c_float, vp, vp]
            L.gemm_s8_zp_noalloc.restype = i32
            L.gemm_s8_zp_workspace_size.argtypes = [i64, i64, i64]
            L.gemm_s8_zp_workspace_size.restype = sz
            L.conv2d_nhwc_f16_implicit.argtypes = [i32] * 11 + [vp, vp, vp, vp, vp]
            L.conv2d_nhwc_f16_implicit.restype = i32
            L.conv2d_nhwc_s8_zp.argtypes = [i32] * 11 + [vp, i32, ctypes.c_int32, vp, i32,
                                                         ctypes.c_int32, vp, vp, vp,
                                                         ctypes.c_float, vp, vp, sz, vp]
            L.conv2d_nhwc_s8_zp.restype = i32
            L.conv2d_nhwc_s8_zp_workspace_size.argtypes = [i32] * 11
            L.conv2d_nhwc_s8_zp_workspace_size.restype = sz
            L.igc_status_string.argtypes = [i32]
            L.igc_status_string.restype = ctypes.c_char_p
            L.igc_check_device_status.argtypes = [vp]
            L.igc_check_device_status.restype = i32
            L.igc_last_device_status.argtypes = []
            L.igc_last_device_status.restype = ctypes.c_uint64
            L.igc_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.igc_set_wait_limit_ns.restype = ctypes.c_uint64
            L.igc_set_tile_width.argtypes = [i32]
            L.igc_set_tile_width.restype = i32
            L.igc_set_stage_depth.argtypes = [i32]
            L.igc_set_stage_depth.restype = i32
            L.igc_set_int8_path.argtypes = [i32]
            L.igc_set_int8_path.restype = i32
            L.igc_plan_gemm.argtypes = [i32, i64, i64, i64, i32, ctypes.POINTER(ctypes.c_int32)]
            L.igc_plan_gemm.restype = i32
            L.igc_debug_wait_timeout_probe.argtypes = [vp]
            L.igc_debug_wait_timeout_probe.restype = i32
            f32 = ctypes.c_float
            L.linear_act.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i32, i32, vp, i64,
                                     vp, i64, vp, i64, i32, vp]
            L.linear_act.restype = i32
            L.linear_act_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64,
                                              vp, i64, vp, i64, vp, i64, i32, vp, i32, vp, sz, vp]
            L.linear_act_backward.restype = i32
            L.gated_ffn.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, i64, vp, vp, i32, i32,
                                    vp, vp, i64, vp, i64, vp]
            L.gated_ffn.restype = i32
            L.gated_ffn_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, i64, i32, vp,
                                             i64, vp, vp, i64, vp, i64, vp, vp, i64, i32, vp, vp,
                                             i32, vp, sz, vp]
            L.gated_ffn_backward.restype = i32
            for name in ("linear_act_backward_workspace_size",
                         "gated_ffn_backward_workspace_size"):
                getattr(L, name).argtypes = [i64, i64, i64]
                getattr(L, name).restype = sz
            L.grad_norm_clip.argtypes = [i64, vp, vp, vp, vp, f32, f32, vp, vp, sz, vp]
            L.grad_norm_clip.restype = i32
            L.grad_norm_clip_workspace_size.argtypes = [i64]
            L.grad_norm_clip_workspace_size.restype = sz
            L.igc_plan_ffn.argtypes = [i32, i64, i64, i64, i32, i32,
                                       ctypes.POINTER(ctypes.c_int32)]
            L.igc_plan_ffn.restype = i32
            L.igc_ffn_cta_resources.argtypes = L.igc_plan_ffn.argtypes
            L.igc_ffn_cta_resources.restype = i32
            f64, u64 = ctypes.c_double, ctypes.c_uint64
            L.dropout_add.argtypes = [i64, i64, vp, i64, i32, vp, i64, f64, u64, u64, vp, vp, i64,
                                      i32, vp]
            L.dropout_add.restype = i32
            L.layer_norm.argtypes = [i64, i64, i32, vp, i64, vp, i64, i32, f64, u64, u64, vp, vp,
                                     vp, i32, f32, vp, i64, vp, i64, vp, vp, vp]
            L.layer_norm.restype = i32
            L.layer_norm_backward.argtypes = [i64, i64, i32, vp, i64, vp, i64, i32, vp, vp, vp,
                                              i32, vp, i64, f64, u64, u64, vp, vp, i64, vp, i64,
                                              vp, vp, i32, vp, sz, vp]
            L.layer_norm_backward.restype = i32
            L.layer_norm_backward_workspace_size.argtypes = [i64, i64]
            L.layer_norm_backward_workspace_size.restype = sz
            L.embedding_lookup.argtypes = [i64, i64, i64, vp, i32, vp, i64, i32, f32, vp, i64, i32,
                                           vp]
            L.embedding_lookup.restype = i32
            L.embedding_backward.argtypes = [i64, i64, i64, vp, i32, vp, i64, i32, f32, i32, vp,
                                             i64, i32, vp, sz, vp]
            L.embedding_backward.restype = i32
            L.embedding_backward_workspace_size.argtypes = [i64, i64, i64]
            L.embedding_backward_workspace_size.restype = sz
            L.igc_version.argtypes = []
            L.igc_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def declared_functions(header: str = HEADER) -> list[str]:
    """Names of the functions a header declares (include/igc.h by default;
    include/igc_debug.h holds the tuning and test hooks)."""
    with open(header) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) -
                  {"sizeof", "defined", "if"})


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _stream(stream):
    """The cudaStream_t handle (as an int) of `stream`, or of the current stream."""
    import torch
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(rc: int, what: str):
    if rc != IGC_OK:
        raise IGCError(rc, what)


def _rows(t, name, dtype=None, shape=None, cuda=True):
    """(rows, cols, row stride in elements) of a 2-D row-major view; checks the
    dtype and, when given, the (rows, cols) shape, then (unless cuda is False,
    for a caller that checks devices last with _require_cuda) the device."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major view with unit inner stride")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if cuda:
        _require_cuda(**{name: t})
    return t.shape[0], t.shape[1], max(t.stride(0), t.shape[1])


def _require_cuda(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")


def _vec(v, name, n, dtype):
    """Checks an optional per-row / per-column vector: dense, `n` elements of
    `dtype` (its device is checked by the caller's _require_cuda)."""
    if v is None:
        return
    if v.dtype != dtype or v.numel() != n or not v.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of length {n}")


def _s8_outputs(C32, C8, M, N):
    """Row strides of the int8 GEMM's outputs (0 for an absent one), shapes checked."""
    import torch
    ldc32 = _rows(C32, "C32", torch.int32, (M, N), cuda=False)[2] if C32 is not None else 0
    ldc8 = _rows(C8, "C8", torch.int8, (M, N), cuda=False)[2] if C8 is not None else 0
    return ldc32, ldc8


def _s8_operands(A, Bt):
    """(M, N, K, lda, ldb) of the int8 GEMM's operands, dtypes and K checked."""
    import torch
    M, K, lda = _rows(A, "A", (torch.uint8, torch.int8), cuda=False)
    N, K2, ldb = _rows(Bt, "Bt", (torch.uint8, torch.int8), cuda=False)
    if K2 != K:
        raise ValueError("A and Bt disagree on K")
    return M, N, K, lda, ldb


def status_string(status: int) -> str:
    return lib().igc_status_string(int(status)).decode()


def igc_status_string(status: int) -> str:
    return status_string(status)


def igc_check_device_status(stream=None) -> int:
    return int(lib().igc_check_device_status(_stream(stream)))


def igc_last_device_status() -> int:
    return int(lib().igc_last_device_status())


# Tuning and test hooks (include/igc_debug.h): thread-local, they force a schedule
# choice of the calling thread's later calls only.

def igc_set_tile_width(bn: int) -> int:
    return int(lib().igc_set_tile_width(int(bn)))


def igc_set_stage_depth(k: int) -> int:
    return int(lib().igc_set_stage_depth(int(k)))


INT8_PATH_TCGEN05, INT8_PATH_MMA_SYNC, INT8_PATH_FUSED, INT8_PATH_CONVERT = 0, 1, 2, 3


def igc_set_int8_path(path: int) -> int:
    return int(lib().igc_set_int8_path(int(path)))


PLAN_GEMM_F16, PLAN_GEMM_BF16, PLAN_GEMM_S8 = 0, 1, 2
_PLAN_FIELDS = ("tile_width", "stage_k", "tiles_m", "tiles_n", "tail_start", "units", "ctas",
                "prefetch_units")


def igc_plan_gemm(op: int, M: int, N: int, K: int, clusters: int = 0) -> dict:
    """The schedule a GEMM call would run with (see include/igc.h); raises on error."""
    out = (ctypes.c_int32 * 8)()
    _check(lib().igc_plan_gemm(int(op), int(M), int(N), int(K), int(clusters), out),
           "igc_plan_gemm")
    return dict(zip(_PLAN_FIELDS, (int(v) for v in out)))


def igc_set_wait_limit_ns(limit_ns: int) -> int:
    return int(lib().igc_set_wait_limit_ns(int(limit_ns)))


def igc_debug_wait_timeout_probe(stream=None) -> int:
    return int(lib().igc_debug_wait_timeout_probe(_stream(stream)))


def igc_version() -> str:
    return lib().igc_version().decode()


# ---------------------------------------------------------------------------
# the three operations
# ---------------------------------------------------------------------------

def gemm_f16(A, Bt, C=None, C_f32_check=None, stream=None):
    """C[i,j] = sum_k A[i,k] Bt[j,k]; A (M,K) fp16, Bt (N,K) fp16 (B column-major),
    C (M,N) fp16 or fp32, C_f32_check optional fp32 (M,N).  Returns C."""
    import torch
    M, K, lda = _rows(A, "A", torch.float16)
    N, K2, ldb = _rows(Bt, "Bt", torch.float16)
    if K2 != K:
        raise ValueError("A and Bt disagree on K")
    if C is None and C_f32_check is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    c_dtype, ldc = IGC_F32, 0
    if C is not None:
        ldc = _rows(C, "C", (torch.float16, torch.float32), (M, N))[2]
        c_dtype = IGC_F16 if C.dtype == torch.float16 else IGC_F32
    ldc32 = 0
    if C_f32_check is not None:
        ldc32 = _rows(C_f32_check, "C_f32_check", torch.float32, (M, N))[2]
    rc = lib().gemm_f16(M, N, K, _ptr(A), lda, _ptr(Bt), ldb, _ptr(C), ldc, c_dtype,
                        _ptr(C_f32_check), ldc32, _stream(stream))
    _check(rc, "gemm_f16")
    return C


def gemm_bf16(A, Bt, C=None, C_f32_check=None, stream=None):
    """C[i,j] = sum_k A[i,k] Bt[j,k]; A (M,K) bf16, Bt (N,K) bf16 (B column-major),
    C (M,N) bf16 or fp32, C_f32_check optional fp32 (M,N).  Returns C."""
    import torch
    M, K, lda = _rows(A, "A", torch.bfloat16)
    N, K2, ldb = _rows(Bt, "Bt", torch.bfloat16)
    if K2 != K:
        raise ValueError("A and Bt disagree on K")
    if C is None and C_f32_check is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    c_dtype, ldc = IGC_F32, 0
    if C is not None:
        ldc = _rows(C, "C", (torch.bfloat16, torch.float32), (M, N))[2]
        c_dtype = IGC_BF16 if C.dtype == torch.bfloat16 else IGC_F32
    ldc32 = 0
    if C_f32_check is not None:
        ldc32 = _rows(C_f32_check, "C_f32_check", torch.float32, (M, N))[2]
    rc = lib().gemm_bf16(M, N, K, _ptr(A), lda, _ptr(Bt), ldb, _ptr(C), ldc, c_dtype,
                         _ptr(C_f32_check), ldc32, _stream(stream))
    _check(rc, "gemm_bf16")
    return C


def gemm_s8_zp_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().gemm_s8_zp_workspace_size(M, N, K))


def gemm_s8_zp(A, Bt, zA=0, zA_row=None, zB=0, zB_col=None, C32=None, C8=None,
               scale=0.0, scale_col=None, workspace=None, stream=None):
    """INT8 GEMM with zero points: A (M,K) uint8/int8, Bt (N,K) uint8/int8.
    Outputs C32 (M,N) int32 and/or C8 (M,N) int8.  Returns (C32, C8)."""
    import torch
    M, N, K, lda, ldb = _s8_operands(A, Bt)
    ldc32, ldc8 = _s8_outputs(C32, C8, M, N)
    _vec(zA_row, "zA_row", M, torch.int32)
    _vec(zB_col, "zB_col", N, torch.int32)
    _vec(scale_col, "scale_col", N, torch.float32)
    _require_cuda(A=A, Bt=Bt, C32=C32, C8=C8, zA_row=zA_row, zB_col=zB_col, scale_col=scale_col)
    need = gemm_s8_zp_workspace_size(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=A.device)
    rc = lib().gemm_s8_zp(M, N, K, _ptr(A), 1 if A.dtype == torch.int8 else 0, lda,
                          _ptr(Bt), 1 if Bt.dtype == torch.int8 else 0, ldb,
                          int(zA), _ptr(zA_row), int(zB), _ptr(zB_col),
                          _ptr(C32), ldc32, _ptr(C8), ldc8, float(scale), _ptr(scale_col),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _stream(stream))
    _check(rc, "gemm_s8_zp")
    return C32, C8


def gemm_s8_zp_dequant(A, Bt, zA=0, zA_row=None, zB=0, zB_col=None, scale_row=None,
                       scale_col=None, bias=None, Y=None, workspace=None, stream=None):
    """INT8 GEMM with zero points and a dequantised fp32 output
    Y = ((fp32(C32) * scale_row_i) * scale_col_j) + bias_j.  Returns Y."""
    import torch
    M, N, K, lda, ldb = _s8_operands(A, Bt)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=A.device)
    ldy = _rows(Y, "Y", torch.float32, (M, N), cuda=False)[2]
    _vec(zA_row, "zA_row", M, torch.int32)
    _vec(zB_col, "zB_col", N, torch.int32)
    _vec(scale_row, "scale_row", M, torch.float32)
    _vec(scale_col, "scale_col", N, torch.float32)
    _vec(bias, "bias", N, torch.float32)
    _require_cuda(A=A, Bt=Bt, Y=Y, zA_row=zA_row, zB_col=zB_col, scale_row=scale_row,
                  scale_col=scale_col, bias=bias)
    if workspace is None:
        workspace = torch.empty(max(gemm_s8_zp_workspace_size(M, N, K), 1), dtype=torch.uint8,
                                device=A.device)
    rc = lib().gemm_s8_zp_dequant(M, N, K, _ptr(A), 1 if A.dtype == torch.int8 else 0, lda,
                                  _ptr(Bt), 1 if Bt.dtype == torch.int8 else 0, ldb,
                                  int(zA), _ptr(zA_row), int(zB), _ptr(zB_col),
                                  _ptr(scale_row), _ptr(scale_col), _ptr(bias), _ptr(Y), ldy,
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check(rc, "gemm_s8_zp_dequant")
    return Y


IGC_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def gemm_s8_zp_noalloc(A, Bt, zA=0, zA_row=None, zB=0, zB_col=None, C32=None, C8=None,
                       scale=0.0, scale_col=None, stream=None):
    """gemm_s8_zp for callers that cannot allocate device memory: the library uses
    its own fixed scratch (IGC_NOALLOC_SCRATCH_BYTES per GPU) instead of a
    workspace.  Calls that overlap on the GPU race on that scratch."""
    import torch
    M, N, K, lda, ldb = _s8_operands(A, Bt)
    ldc32, ldc8 = _s8_outputs(C32, C8, M, N)
    _vec(zA_row, "zA_row", M, torch.int32)
    _vec(zB_col, "zB_col", N, torch.int32)
    _vec(scale_col, "scale_col", N, torch.float32)
    _require_cuda(A=A, Bt=Bt, C32=C32, C8=C8, zA_row=zA_row, zB_col=zB_col, scale_col=scale_col)
    rc = lib().gemm_s8_zp_noalloc(M, N, K, _ptr(A), 1 if A.dtype == torch.int8 else 0, lda,
                                  _ptr(Bt), 1 if Bt.dtype == torch.int8 else 0, ldb,
                                  int(zA), _ptr(zA_row), int(zB), _ptr(zB_col),
                                  _ptr(C32), ldc32, _ptr(C8), ldc8, float(scale), _ptr(scale_col),
                                  _stream(stream))
    _check(rc, "gemm_s8_zp_noalloc")
    return C32, C8


def gemm_s8_zp_prepare(A, Bt, workspace, M=None, N=None, K=None, stream=None):
    """Operand pre-pass of gemm_s8_zp into `workspace`; A or Bt may be None to keep
    the prepared copy of that operand (M, N, K must then be given)."""
    import torch
    lda = ldb = 0
    a_signed = b_signed = 0
    if A is not None:
        M, K, lda = _rows(A, "A", (torch.uint8, torch.int8))
        a_signed = 1 if A.dtype == torch.int8 else 0
    if Bt is not None:
        N, K2, ldb = _rows(Bt, "Bt", (torch.uint8, torch.int8))
        if K is not None and K2 != K:
            raise ValueError("A and Bt disagree on K")
        K = K2
        b_signed = 1 if Bt.dtype == torch.int8 else 0
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    rc = lib().gemm_s8_zp_prepare(M, N, K, _ptr(A), a_signed, lda, _ptr(Bt), b_signed, ldb,
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check(rc, "gemm_s8_zp_prepare")


def gemm_s8_zp_run(M, N, K, a_signed, b_signed, workspace, zA=0, zA_row=None, zB=0, zB_col=None,
                   C32=None, C8=None, scale=0.0, scale_col=None, stream=None):
    """tcgen05 GEMM + fused zero-point correction / requantisation over a prepared workspace."""
    import torch
    M, N, K = int(M), int(N), int(K)
    ldc32, ldc8 = _s8_outputs(C32, C8, M, N)
    _vec(zA_row, "zA_row", M, torch.int32)
    _vec(zB_col, "zB_col", N, torch.int32)
    _vec(scale_col, "scale_col", N, torch.float32)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _require_cuda(C32=C32, C8=C8, zA_row=zA_row, zB_col=zB_col, scale_col=scale_col,
                  workspace=workspace)
    rc = lib().gemm_s8_zp_run(M, N, K, int(a_signed), int(b_signed), int(zA), _ptr(zA_row),
                              int(zB), _ptr(zB_col), _ptr(C32), ldc32, _ptr(C8), ldc8,
                              float(scale), _ptr(scale_col), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "gemm_s8_zp_run")
    return C32, C8


def conv2d_nhwc_f16_implicit(x, w, y=None, y_f32_check=None, pad=(1, 1), stride=(1, 1),
                             stream=None):
    """y[n,p,q,k] = sum_{r,s,c} xpad[n, p*sh+r-ph, q*sw+s-pw, c] * w[k,r,s,c];
    x NHWC fp16, w KRSC fp16, y NPQK fp16.  Returns y (or y_f32_check if y is None)."""
    import torch
    if x.dim() != 4 or w.dim() != 4 or x.dtype != torch.float16 or w.dtype != torch.float16:
        raise ValueError("x and w must be 4-D fp16 tensors")
    if not (x.is_contiguous() and w.is_contiguous() and x.is_cuda and w.is_cuda):
        raise ValueError("x and w must be dense CUDA tensors")
    N, H, W, C = x.shape
    K, R, S, C2 = w.shape
    if C2 != C:
        raise ValueError("x and w disagree on C")
    ph, pw = pad
    sh, sw = stride
    P = (H + 2 * ph - R) // sh + 1
    Q = (W + 2 * pw - S) // sw + 1
    if y is None and y_f32_check is None:
        y = torch.empty((N, P, Q, K), dtype=torch.float16, device=x.device)
    for t, dt, name in ((y, torch.float16, "y"), (y_f32_check, torch.float32, "y_f32_check")):
        if t is not None and (tuple(t.shape) != (N, P, Q, K) or t.dtype != dt or not t.is_contiguous()):
            raise ValueError(f"{name} must be a dense ({N},{P},{Q},{K}) {dt} tensor")
    rc = lib().conv2d_nhwc_f16_implicit(N, H, W, C, K, R, S, ph, pw, sh, sw, _ptr(x), _ptr(w),
                                        _ptr(y), _ptr(y_f32_check), _stream(stream))
    _check(rc, "conv2d_nhwc_f16_implicit")
    return y if y is not None else y_f32_check


def conv2d_nhwc_s8_zp_workspace_size(N, H, W, C, K, R, S, pad=(1, 1), stride=(1, 1)) -> int:
    return int(lib().conv2d_nhwc_s8_zp_workspace_size(N, H, W, C, K, R, S, pad[0], pad[1],
                                                      stride[0], stride[1]))


def conv2d_nhwc_s8_zp(x, w, zX, zW=0, zW_k=None, y32=None, y8=None, scale=0.0, scale_k=None,
                      pad=(1, 1), stride=(1, 1), workspace=None, stream=None):
    """INT8 convolution with zero points (padding value zX): x NHWC uint8/int8,
    w KRSC uint8/int8; outputs y32 (int32) and/or y8 (int8), NPQK.  Returns (y32, y8)."""
    import torch
    for t, name in ((x, "x"), (w, "w")):
        if t.dim() != 4 or t.dtype not in (torch.uint8, torch.int8) or not t.is_contiguous() \
                or not t.is_cuda:
            raise ValueError(f"{name} must be a dense 4-D CUDA uint8/int8 tensor")
    N, H, W, C = x.shape
    K, R, S, C2 = w.shape
    if C2 != C:
        raise ValueError("x and w disagree on C")
    P = (H + 2 * pad[0] - R) // stride[0] + 1
    Q = (W + 2 * pad[1] - S) // stride[1] + 1
    for t, dt, name in ((y32, torch.int32, "y32"), (y8, torch.int8, "y8")):
        if t is not None and (tuple(t.shape) != (N, P, Q, K) or t.dtype != dt or not t.is_contiguous()):
            raise ValueError(f"{name} must be a dense ({N},{P},{Q},{K}) {dt} tensor")
    for v, name, dt in ((zW_k, "zW_k", torch.int32), (scale_k, "scale_k", torch.float32)):
        if v is not None and (v.dtype != dt or v.numel() != K or not v.is_contiguous() or not v.is_cuda):
            raise ValueError(f"{name} must be a contiguous CUDA {dt} vector of length {K}")
    if workspace is None:
        need = conv2d_nhwc_s8_zp_workspace_size(N, H, W, C, K, R, S, pad, stride)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    rc = lib().conv2d_nhwc_s8_zp(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1],
                                 _ptr(x), 1 if x.dtype == torch.int8 else 0, int(zX),
                                 _ptr(w), 1 if w.dtype == torch.int8 else 0, int(zW), _ptr(zW_k),
                                 _ptr(y32), _ptr(y8), float(scale), _ptr(scale_k),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(rc, "conv2d_nhwc_s8_zp")
    return y32, y8


# ---------------------------------------------------------------------------
# feed-forward operators (include/igc_ffn.h)
#
# None of them takes part in autograd: results carry no history, also of tensors that
# require a gradient; the *_backward functions are called for the gradients.
# ---------------------------------------------------------------------------

_ACTS = {"none": IGC_ACT_NONE, "relu": IGC_ACT_RELU, "gelu": IGC_ACT_GELU,
         "gelu_tanh": IGC_ACT_GELU_TANH, "silu": IGC_ACT_SILU}
_dtype_codes = {}


def _dtype_code(dtype):
    """IGC_F32 / IGC_F16 / IGC_BF16 of a torch dtype, None for any other."""
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float32: IGC_F32, torch.float16: IGC_F16,
                             torch.bfloat16: IGC_BF16})
    return _dtype_codes.get(dtype)


def _operand_code(t, name):
    code = _dtype_code(t.dtype)
    if code is None or code == IGC_F32:
        raise TypeError(f"{name} has dtype {t.dtype}: fp16 or bf16 is needed")
    return code


def _act_code(act):
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act is {act!r}: one of {', '.join(_ACTS)}") from None


def _mat(t, name, dtypes, rows, cols, dev):
    """(pointer, row stride in elements) of a rows x cols matrix: unit inner stride, rows
    that do not overlap (so no broadcast view), one of `dtypes`, on device `dev`.  A single
    row has no stride of its own: it gets one that suits TMA.  (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or (s0 < cols and rows > 1):
        raise ValueError(f"{name} must be row-major with unit inner stride and rows apart")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    return t.data_ptr(), s0 if rows > 1 else (cols + 7) // 8 * 8


def _vector(v, name, dtypes, n, dev):
    """(pointer, dtype code) of an optional vector of n elements ((None, IGC_F32) for None)."""
    if v is None:
        return None, IGC_F32
    if v.dtype not in dtypes or v.shape != (n,) or not v.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of length {n} and type "
                         f"{' or '.join(str(d) for d in dtypes)}")
    if v.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    return v.data_ptr(), _dtype_code(v.dtype)


def _two_dims(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _check_device(dev, name):
    """The device that all tensors of a call are on must be the current CUDA device."""
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _torch()._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _handle(stream, dev):
    """The cudaStream_t handle of `stream`, or of device dev's current stream."""
    return _torch()._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _new(shape, dtype, device, stream):
    """An uninitialised tensor that is safe to use on `stream` (None: the current one):
    memory that the caching allocator hands out belongs to the stream it was asked on."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# Workspaces up to this size are kept for the next call of the same thread on the default
# stream (asking the allocator for one costs 3 to 6 us of host time in calls that take about
# 20); larger ones go back to the allocator when the call returns.  Only the default stream's:
# it is never destroyed, so its handle cannot come to name another stream, and a thread keeps
# one workspace per device however many streams it uses.
_KEPT_WORKSPACE_BYTES = 32 * 1024 * 1024


class _Kept:
    """A thread's workspace for the default stream of each device."""

    def __init__(self):
        self.by_device = {}
        with _lock:
            _all_kept.add(self)


_thread = threading.local()
_all_kept = weakref.WeakSet()


def release_workspaces():
    """Gives the workspaces that the binding keeps between calls (at most 32 MB per thread
    and device) back to torch's allocator, those of every thread; later calls get new ones."""
    with _lock:
        for kept in _all_kept:
            kept.by_device.clear()


def _workspace(workspace, need, like, stream):
    """The workspace of a call: the one given, the one that this thread keeps for the default
    stream, or a new one.  Calls on one stream use it in stream order; another thread's
    calls, which could come between a call's launches, have their own.  A call on any other
    stream and one under graph capture (the graph goes on using it) get a new one."""
    torch = _torch()
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        if workspace.get_device() != like.get_device():
            raise ValueError("workspace is on another device")
        return workspace
    need = max(need, 1)
    dev = like.get_device()
    if stream is not None or need > _KEPT_WORKSPACE_BYTES or _handle(None, dev) != 0 or \
            torch.cuda.is_current_stream_capturing():
        return _new((need,), torch.uint8, like.device, stream)
    try:
        by_device = _thread.kept.by_device
    except AttributeError:
        _thread.kept = _Kept()
        by_device = _thread.kept.by_device
    kept = by_device.get(dev)
    if kept is None or kept.numel() < need:
        kept = by_device[dev] = _new((need,), torch.uint8, like.device, None)
    return kept


def linear_act(X, W, bias=None, act="none", residual=None, Y=None, Z=None, stream=None):
    """Y = act(X W^T + bias) + residual; X (M,K), W (N,K), residual and Z (M,N) of one
    type (fp16 or bf16), Y (M,N) of that type or fp32, bias (N) of that type or fp32.
    Z, if given, receives the pre-activation for linear_act_backward, which is to be
    called for the gradients: the result has no autograd history.  residual may be Y
    itself.  Returns Y (allocated if None)."""
    dtype = X.dtype
    dt = _operand_code(X, "X")
    code = _act_code(act)
    M, K = _two_dims(X, "X")
    N = _two_dims(W, "W")[0]
    dev = X.get_device()
    own, either = (dtype,), (dtype, _torch().float32)
    x, ldx = _mat(X, "X", own, M, K, dev)
    w, ldw = _mat(W, "W", own, N, K, dev)
    r, ldr = _mat(residual, "residual", own, M, N, dev)
    z, ldz = _mat(Z, "Z", own, M, N, dev)
    b, bt = _vector(bias, "bias", either, N, dev)
    y, ldy = _mat(Y, "Y", either, M, N, dev)
    _check_device(dev, "X")
    if Y is None:
        Y = _new((M, N), dtype, X.device, stream)
        y, ldy = Y.data_ptr(), N
    _check(lib().linear_act(M, N, K, dt, x, ldx, w, ldw, b, bt, code, r, ldr, z, ldz, y, ldy,
                            dt if Y.dtype is dtype else IGC_F32, _handle(stream, dev)),
           "linear_act")
    return Y


def linear_act_backward_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().linear_act_backward_workspace_size(M, N, K))


def linear_act_backward(dY, X, W, act="none", Z=None, dX=None, dW=None, dbias=None,
                        workspace=None, stream=None):
    """Gradients of linear_act from dY (M,N) and the pre-activation Z (M,N) that it kept
    (not needed without an activation): dX (M,K), dW (N,K), dbias (N).  The ones given
    are computed (X is needed for dW, W for dX; the other may be None); with none
    given, dX and dW are allocated.  dW and dbias may be fp32.  No tensor's .grad is
    touched.  Returns (dX, dW, dbias)."""
    dtype = dY.dtype
    dt = _operand_code(dY, "dY")
    code = _act_code(act)
    M, N = _two_dims(dY, "dY")
    dev = dY.get_device()
    if dX is None and dW is None and dbias is None:
        if X is None or W is None:
            raise ValueError("X and W are needed for dX and dW")
        dX = _new(X.shape, dtype, dY.device, stream)
        dW = _new(W.shape, dtype, dY.device, stream)
    if (dX is not None and W is None) or (dW is not None and X is None):
        raise ValueError("dX needs W and dW needs X")
    if code != IGC_ACT_NONE and Z is None:
        raise ValueError("Z, the pre-activation, is needed with an activation")
    k_of = W if W is not None else X
    K = _two_dims(k_of, "W" if W is not None else "X")[1] if k_of is not None else 0
    own, either = (dtype,), (dtype, _torch().float32)
    dy, lddy = _mat(dY, "dY", own, M, N, dev)
    z, ldz = _mat(Z, "Z", own, M, N, dev)
    x, ldx = _mat(X, "X", own, M, K, dev)
    w, ldw = _mat(W, "W", own, N, K, dev)
    dx, lddx = _mat(dX, "dX", own, M, K, dev)
    dw, lddw = _mat(dW, "dW", either, N, K, dev)
    db, bt = _vector(dbias, "dbias", either, N, dev)
    _check_device(dev, "dY")
    L = lib()
    ws = _workspace(workspace, L.linear_act_backward_workspace_size(M, N, K), dY, stream)
    _check(L.linear_act_backward(M, N, K, dt, dy, lddy, z, ldz, code, x, ldx, w, ldw, dx, lddx,
                                 dw, lddw, IGC_F32 if dW is None else _dtype_code(dW.dtype), db,
                                 bt, ws.data_ptr(), ws.numel(), _handle(stream, dev)),
           "linear_act_backward")
    return dX, dW, dbias


def _one_stride(a, b, names):
    if a != b:
        raise ValueError(f"{names} must have one row stride")


def gated_ffn(X, Wg, Wu, bg=None, bu=None, act="silu", H=None, G=None, U=None, stream=None):
    """H = act(X Wg^T + bg) * (X Wu^T + bu); X (M,K), Wg and Wu (F,K) with one row stride
    (two matrices, or the halves of a (2F,K) one), H (M,F), all of one type (fp16 or
    bf16); bg and bu (F) of that type or fp32.  G and U, if given, receive the two
    pre-activations for gated_ffn_backward, which is to be called for the gradients: the
    result has no autograd history.  Returns H (allocated if None)."""
    dtype = X.dtype
    dt = _operand_code(X, "X")
    code = _act_code(act)
    M, K = _two_dims(X, "X")
    F = _two_dims(Wg, "Wg")[0]
    dev = X.get_device()
    own, either = (dtype,), (dtype, _torch().float32)
    if (G is None) != (U is None):
        raise ValueError("G and U go together")
    x, ldx = _mat(X, "X", own, M, K, dev)
    wg, ldw = _mat(Wg, "Wg", own, F, K, dev)
    wu, ldwu = _mat(Wu, "Wu", own, F, K, dev)
    _one_stride(ldw, ldwu, "Wg and Wu")
    h, ldh = _mat(H, "H", own, M, F, dev)
    g, ldg = _mat(G, "G", own, M, F, dev)
    u, ldu = _mat(U, "U", own, M, F, dev)
    _one_stride(ldg, ldu, "G and U")
    b0, bt0 = _vector(bg, "bg", either, F, dev)
    b1, bt1 = _vector(bu, "bu", either, F, dev)
    if bg is not None and bu is not None and bt0 != bt1:
        raise ValueError("bg and bu must have one type")
    _check_device(dev, "X")
    if H is None:
        H = _new((M, F), dtype, X.device, stream)
        h, ldh = H.data_ptr(), F
    _check(lib().gated_ffn(M, F, K, dt, x, ldx, wg, wu, ldw, b0, b1, bt0 if bg is not None else bt1,
                           code, g, u, ldg, h, ldh, _handle(stream, dev)), "gated_ffn")
    return H


def gated_ffn_backward_workspace_size(M: int, F: int, K: int) -> int:
    return int(lib().gated_ffn_backward_workspace_size(M, F, K))


def gated_ffn_backward(dH, G, U, X, Wg, Wu, act="silu", dX=None, dWg=None, dWu=None, dbg=None,
                       dbu=None, workspace=None, stream=None):
    """Gradients of gated_ffn from dH (M,F) and the pre-activations G and U (M,F) that it
    kept: dX (M,K), dWg and dWu (F,K), dbg and dbu (F).  The ones given are computed
    (the pairs go together; X is needed for the weights', Wg and Wu for dX); with none
    given, dX, dWg and dWu are allocated.  The weights' and biases' may be fp32.  No
    tensor's .grad is touched.  Returns (dX, dWg, dWu, dbg, dbu)."""
    dtype = dH.dtype
    dt = _operand_code(dH, "dH")
    code = _act_code(act)
    M, F = _two_dims(dH, "dH")
    dev = dH.get_device()
    if (Wg is None) != (Wu is None) or (dWg is None) != (dWu is None) or \
            (dbg is None) != (dbu is None):
        raise ValueError("Wg and Wu, dWg and dWu, and dbg and dbu go together")
    if dX is None and dWg is None and dbg is None:
        if X is None or Wg is None:
            raise ValueError("X, Wg and Wu are needed for dX, dWg and dWu")
        dX = _new(X.shape, dtype, dH.device, stream)
        dWg = _new(Wg.shape, dtype, dH.device, stream)
        dWu = _new(Wg.shape, dtype, dH.device, stream)
    if (dX is not None and Wg is None) or (dWg is not None and X is None):
        raise ValueError("dX needs Wg and Wu, dWg and dWu need X")
    k_of = Wg if Wg is not None else X
    K = _two_dims(k_of, "Wg" if Wg is not None else "X")[1] if k_of is not None else 0
    own, either = (dtype,), (dtype, _torch().float32)
    dh, lddh = _mat(dH, "dH", own, M, F, dev)
    g, ldg = _mat(G, "G", own, M, F, dev)
    u, ldu = _mat(U, "U", own, M, F, dev)
    _one_stride(ldg, ldu, "G and U")
    x, ldx = _mat(X, "X", own, M, K, dev)
    wg, ldw = _mat(Wg, "Wg", own, F, K, dev)
    wu, ldwu = _mat(Wu, "Wu", own, F, K, dev)
    _one_stride(ldw, ldwu, "Wg and Wu")
    dx, lddx = _mat(dX, "dX", own, M, K, dev)
    dwg, lddw = _mat(dWg, "dWg", either, F, K, dev)
    dwu, lddwu = _mat(dWu, "dWu", either if dWg is None else (dWg.dtype,), F, K, dev)
    _one_stride(lddw, lddwu, "dWg and dWu")
    b0, bt = _vector(dbg, "dbg", either, F, dev)
    b1, bt1 = _vector(dbu, "dbu", either, F, dev)
    if bt != bt1:
        raise ValueError("dbg and dbu must have one type")
    _check_device(dev, "dH")
    L = lib()
    ws = _workspace(workspace, L.gated_ffn_backward_workspace_size(M, F, K), dH, stream)
    _check(L.gated_ffn_backward(M, F, K, dt, dh, lddh, g, u, ldg, code, x, ldx, wg, wu, ldw, dx,
                                lddx, dwg, dwu, lddw,
                                IGC_F32 if dWg is None else _dtype_code(dWg.dtype), b0, b1, bt,
                                ws.data_ptr(), ws.numel(), _handle(stream, dev)),
           "gated_ffn_backward")
    return dX, dWg, dWu, dbg, dbu


PLAN_FFN_LINEAR, PLAN_FFN_GATED, PLAN_FFN_GRAD_X, PLAN_FFN_GRAD_W = 0, 1, 2, 3
_PLAN_FFN_FIELDS = ("small", "rows", "row_blocks", "columns", "split", "small_ns", "tiles_ns")


def igc_plan_ffn(op: int, M: int, N: int, K: int, count: int = 1, sms: int = 152) -> dict:
    """The schedule that a feed-forward product runs with (see include/igc_ffn.h)."""
    out = (ctypes.c_int32 * 7)()
    _check(lib().igc_plan_ffn(int(op), int(M), int(N), int(K), int(count), int(sms), out),
           "igc_plan_ffn")
    return dict(zip(_PLAN_FFN_FIELDS, (int(v) for v in out)))


def _ffn_cta_resources(op: int, M: int, N: int, K: int, count: int = 1, sms: int = 152):
    """(tensor-memory columns, bytes of dynamic shared memory) of a CTA of the kernel that
    igc_plan_ffn answers."""
    out = (ctypes.c_int32 * 2)()
    _check(lib().igc_ffn_cta_resources(int(op), int(M), int(N), int(K), int(count), int(sms),
                                       out), "igc_ffn_cta_resources")
    return int(out[0]), int(out[1])


def grad_norm_clip_workspace_size(count: int) -> int:
    return int(lib().grad_norm_clip_workspace_size(int(count)))


def grad_norm_clip(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None, stream=None):
    """Clips the global 2-norm of `grads` (a sequence of contiguous fp32, fp16 or bf16
    tensors, types may differ): each becomes g * min(1, max_norm / (norm + eps)), in place
    or in `out` (tensors of the same sizes and types).  out=False: the norm alone.
    Returns the norm, a one-element fp32 CUDA tensor (`norm`, or allocated); nothing
    waits for the GPU."""
    import torch
    T = torch.Tensor
    grads = list(grads)
    n = len(grads)
    if out is None or out is False:
        every = grads
    else:
        every = grads + list(out)
        if len(every) != 2 * n:
            raise ValueError("out must have as many tensors as grads")
    dtypes = [g.dtype for g in every]
    codes = [_dtype_code(t) for t in dtypes[:n]]
    if None in codes:
        raise TypeError(f"a gradient has dtype {dtypes[codes.index(None)]}")
    sizes = list(map(T.numel, every))
    if not all(map(T.is_contiguous, every)):
        raise ValueError("gradients and out must be contiguous")
    devices = set(map(T.get_device, every))
    if -1 in devices:
        raise ValueError("gradients and out must be CUDA tensors")
    if len(devices) > 1:
        raise ValueError("gradients and out must be on one device")
    if len(every) > n and (dtypes[:n] != dtypes[n:] or sizes[:n] != sizes[n:]):
        raise ValueError("out must match grads in type and size")
    ptrs = array.array("Q", map(T.data_ptr, every))
    g_ptr = ptrs.buffer_info()[0]
    o_ptr = None if out is False else (g_ptr if out is None else g_ptr + 8 * n)
    sizes, codes = array.array("q", sizes[:n]), array.array("i", codes)
    if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1 or
                             not norm.is_cuda):
        raise ValueError("norm must be a one-element fp32 CUDA tensor")
    device = grads[0].device if n else (norm.device if norm is not None else "cuda")
    if norm is None:
        norm = _new((), torch.float32, device, stream)
    dev = norm.get_device()
    if n and dev not in devices:
        raise ValueError("norm is on another device")
    _check_device(dev, "norm")
    ws = _workspace(workspace, grad_norm_clip_workspace_size(n), norm, stream)
    rc = lib().grad_norm_clip(n, g_ptr, sizes.buffer_info()[0], codes.buffer_info()[0], o_ptr,
                              float(max_norm), float(eps), norm.data_ptr(), ws.data_ptr(),
                              ws.numel(), _handle(stream, dev))
    _check(rc, "grad_norm_clip")
    return norm


# ---------------------------------------------------------------------------
# embedding, layer norm and dropout (include/igc_layers.h)
#
# As the feed-forward operators they take no part in autograd: the *_backward functions are
# called for the gradients (that of dropout_add is dropout_add on the gradient).
# ---------------------------------------------------------------------------

def _type_code(t, name):
    code = _dtype_code(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}: fp32, fp16 or bf16 is needed")
    return code


def _new_rows(rows, cols, dtype, like, stream):
    """An uninitialised rows x cols matrix and its row stride.  Its rows follow one another closely
    unless those of `like`, the call's input, are padded so that each starts on a 16-byte boundary:
    then so are these, or the result's alone would send the call to the slow kernels."""
    size, step = dtype.itemsize, like.stride(0) * like.element_size()
    if cols * size % 16 == 0 or rows < 2 or like.shape[0] < 2 or step % 16 != 0 or \
            like.data_ptr() % 16 != 0:
        return _new((rows, cols), dtype, like.device, stream), cols
    ld = -(-cols * size // 16) * 16 // size
    return _new((rows, ld), dtype, like.device, stream)[:, :cols], ld


_or_f32 = {}


def _type_or_f32(dtype):
    """(dtype, fp32), of which dtype may be the one."""
    types = _or_f32.get(dtype)
    if types is None:
        f32 = _torch().float32
        types = _or_f32[dtype] = (dtype,) if dtype is f32 else (dtype, f32)
    return types


def _drop_args(p, seed, offset, step, dev):
    """(p, seed, offset, pointer of step) of a call with dropout."""
    if p == 0.0 and seed is None and step is None and offset == 0:
        return 0.0, 0, 0, None
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p is {p}: a probability is needed")
    if seed is None:
        if p > 0.0:
            raise ValueError("seed is needed with p > 0")
        seed = 0
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset must be in [0, 2^64)")
    if step is None:
        return p, seed, offset, None
    if step.dtype != _torch().int64 or step.numel() != 1:
        raise ValueError("step must be a one-element int64 tensor")
    if step.get_device() != dev:
        raise ValueError("step is on another device")
    return p, seed, offset, step.data_ptr()


def _floats(v, name, n, dev):
    """Pointer of an optional fp32 vector of n elements."""
    return None if v is None else _vector(v, name, (_torch().float32,), n, dev)[0]


def dropout_add(X, p, seed=None, offset=0, step=None, residual=None, Y=None, stream=None):
    """Y = residual + drop(X): each element of X (M,N) is kept and scaled with probability
    1 - p (to a multiple of 1/65536), else 0.  Which ones follows from (seed, offset, row,
    column) and is computed again where it is needed, never stored.  step, a one-element int64
    CUDA tensor, is added to offset when the kernel runs (for captured graphs).  Calls are
    independent where (seed, offset + step) differ: layers that share a seed and have offsets 0,
    1, 2, ... repeat one another's masks a step later, so give each a seed of its own.  X, Y and residual (M,N) fp32, fp16 or bf16;
    residual has Y's type, which is X's unless one of them is fp32.  Y may be X or residual.
    The gradient of X is dropout_add(dY, p, seed, offset, step), that of residual dY.
    Returns Y (allocated if None, of residual's type, else X's; its rows are padded to 16 bytes
    where X's are)."""
    xt = _type_code(X, "X")
    M, N = _two_dims(X, "X")
    dev = X.get_device()
    like = Y if Y is not None else (residual if residual is not None else X)
    yt = _type_code(like, "Y" if like is Y else "residual")
    if xt != yt and xt != IGC_F32 and yt != IGC_F32:
        raise TypeError(f"X has dtype {X.dtype}, the output {like.dtype}")
    x, ldx = _mat(X, "X", (X.dtype,), M, N, dev)
    r, ldr = _mat(residual, "residual", (like.dtype,), M, N, dev)
    y, ldy = _mat(Y, "Y", (like.dtype,), M, N, dev)
    p, seed, offset, step = _drop_args(p, seed, offset, step, dev)
    _check_device(dev, "X")
    if Y is None:
        Y, ldy = _new_rows(M, N, like.dtype, X, stream)
        y = Y.data_ptr()
    _check(lib().dropout_add(M, N, x, ldx, xt, r, ldr, p, seed, offset, step, y, ldy, yt,
                             _handle(stream, dev)), "dropout_add")
    return Y


def layer_norm(X, w=None, b=None, eps=1e-5, residual=None, p=0.0, seed=None, offset=0, step=None,
               Y=None, S=None, mean=None, rstd=None, stream=None):
    """S = residual + drop(X) and Y = (S - mean) rstd w + b over the rows of S, in one pass.
    X and Y (M,N) of one type (fp32, fp16 or bf16), residual and S (M,N) of that type or
    fp32, w and b (N) of that type or fp32.  Dropout (p, seed, offset, step) as in
    dropout_add.  Without residual and dropout S is X, which may then be fp32 whatever Y is.
    S, mean and rstd (M, fp32), if given, receive what layer_norm_backward needs, which is to
    be called for the gradients: the result has no autograd history.  S may be residual
    itself.  Returns Y (allocated if None, of X's type, its rows padded to 16 bytes where X's
    are)."""
    M, N = _two_dims(X, "X")
    _type_code(X, "X")
    dev = X.get_device()
    dtype = X.dtype if Y is None else Y.dtype
    dt = _dtype_code(dtype)
    if dt is None:
        raise TypeError(f"Y has dtype {dtype}: fp32, fp16 or bf16 is needed")
    own, either = (dtype,), _type_or_f32(dtype)
    drop = _drop_args(p, seed, offset, step, dev)
    if residual is None and drop[0] == 0.0:
        x, ldx = None, 0
        r, ldr = _mat(X, "X", either, M, N, dev)      # the stream itself
        s_dtype = X.dtype
    else:
        x, ldx = _mat(X, "X", own, M, N, dev)
        r, ldr = _mat(residual, "residual", either, M, N, dev)
        s_dtype = residual.dtype if residual is not None else (dtype if S is None else S.dtype)
    s, lds = _mat(S, "S", either if residual is None and x is not None else (s_dtype,), M, N, dev)
    y, ldy = _mat(Y, "Y", own, M, N, dev)
    wp, wt = _vector(w, "w", either, N, dev)
    bp, bt = _vector(b, "b", either, N, dev)
    if w is not None and b is not None and wt != bt:
        raise ValueError("w and b must have one type")
    m, rs = _floats(mean, "mean", M, dev), _floats(rstd, "rstd", M, dev)
    _check_device(dev, "X")
    if Y is None:
        Y, ldy = _new_rows(M, N, dtype, X, stream)
        y = Y.data_ptr()
    _check(lib().layer_norm(M, N, dt, x, ldx, r, ldr, _dtype_code(s_dtype), *drop, wp, bp,
                            wt if w is not None else bt, float(eps), s, lds, y, ldy, m, rs,
                            _handle(stream, dev)), "layer_norm")
    return Y


def layer_norm_backward_workspace_size(M: int, N: int) -> int:
    return int(lib().layer_norm_backward_workspace_size(M, N))


def layer_norm_backward(dY, S, mean, rstd, w=None, dS_add=None, p=0.0, seed=None, offset=0,
                        step=None, dS=None, dX=None, dw=None, db=None, workspace=None,
                        stream=None):
    """Gradients of layer_norm from dY (M,N) and the S (M,N), mean and rstd (M) that it kept:
    dS (M,N), that of S and so of the residual, with dS_add (the gradient that reaches S past
    the norm) added; dX (M,N), that of X, through the dropout of the same (p, seed, offset,
    step); dw and db (N).  The ones given are computed; with none given, dS, dw and db are
    allocated (dw and db in fp32, dS with rows padded to 16 bytes where S's are).  dX has dY's type; S, dS_add and dS are of that type or
    fp32, all the same; w, dw and db of dY's type or fp32.  dS may be dS_add itself.  No
    tensor's .grad is touched.  Returns (dS, dX, dw, db)."""
    dt = _type_code(dY, "dY")
    M, N = _two_dims(dY, "dY")
    dev = dY.get_device()
    torch = _torch()
    drop = _drop_args(p, seed, offset, step, dev)
    own, either = (dY.dtype,), _type_or_f32(dY.dtype)
    y, ldy = _mat(dY, "dY", own, M, N, dev)
    s, lds = _mat(S, "S", either, M, N, dev)
    stream_type = (S.dtype,)
    a, lda = _mat(dS_add, "dS_add", stream_type, M, N, dev)
    m, rs = _floats(mean, "mean", M, dev), _floats(rstd, "rstd", M, dev)
    if m is None or rs is None:
        raise ValueError("mean and rstd are needed")
    wp, wt = _vector(w, "w", either, N, dev)
    if dS is None and dX is None and dw is None and db is None:
        dS, _ = _new_rows(M, N, S.dtype, S, stream)
        dw, db = (_new((N,), torch.float32, dY.device, stream) for _ in range(2))
    ds, ldds = _mat(dS, "dS", stream_type, M, N, dev)
    dx, lddx = _mat(dX, "dX", own, M, N, dev)
    dwp, dwt = _vector(dw, "dw", either, N, dev)
    dbp, dbt = _vector(db, "db", either, N, dev)
    if dw is not None and db is not None and dwt != dbt:
        raise ValueError("dw and db must have one type")
    _check_device(dev, "dY")
    L = lib()
    ws, n = None, 0
    if dw is not None or db is not None:
        ws = _workspace(workspace, L.layer_norm_backward_workspace_size(M, N), dY, stream)
        ws, n = ws.data_ptr(), ws.numel()
    _check(L.layer_norm_backward(M, N, dt, y, ldy, s, lds, _dtype_code(S.dtype), m, rs, wp, wt, a,
                                 lda, *drop, ds, ldds, dx, lddx, dwp, dbp,
                                 dwt if dw is not None else dbt, ws, n, _handle(stream, dev)),
           "layer_norm_backward")
    return dS, dX, dw, db


def _tokens(tokens, dev):
    """(pointer, length, bytes of an element) of a vector of token ids."""
    torch = _torch()
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"tokens has dtype {tokens.dtype}: int32 or int64 is needed")
    if tokens.dim() != 1 or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous vector")
    if tokens.get_device() != dev:
        raise ValueError("tokens is on another device")
    return tokens.data_ptr(), tokens.shape[0], tokens.element_size()


def embedding_lookup(tokens, W, scale=1.0, Y=None, stream=None):
    """Y[i] = scale W[tokens[i]]: tokens (M) int32 or int64, W (V,D) fp32, fp16 or bf16, Y (M,D)
    of that type or fp32.  A token outside [0, V) gives a row of zeros.  The result has no
    autograd history (embedding_backward).  Returns Y (allocated if None, of W's type, its rows
    padded to 16 bytes where W's are)."""
    wt = _type_code(W, "W")
    V, D = _two_dims(W, "W")
    dev = W.get_device()
    tp, M, size = _tokens(tokens, dev)
    w, ldw = _mat(W, "W", (W.dtype,), V, D, dev)
    y, ldy = _mat(Y, "Y", _type_or_f32(W.dtype), M, D, dev)
    _check_device(dev, "W")
    if Y is None:
        Y, ldy = _new_rows(M, D, W.dtype, W, stream)
        y = Y.data_ptr()
    _check(lib().embedding_lookup(M, V, D, tp, size, w, ldw, wt, float(scale), y, ldy,
                                  _dtype_code(Y.dtype), _handle(stream, dev)),
           "embedding_lookup")
    return Y


def embedding_backward_workspace_size(M: int, V: int, D: int) -> int:
    return int(lib().embedding_backward_workspace_size(M, V, D))


def embedding_backward(tokens, dY, V=None, scale=1.0, dW=None, accumulate=False, workspace=None,
                       stream=None):
    """dW[v] = scale * sum of dY[i] over the positions i with tokens[i] = v: dY (M,D) fp32, fp16
    or bf16, dW (V,D) of that type or fp32 (allocated in dY's type for V rows if None, padded to
    16 bytes where dY's are).  All of dW is written, or with accumulate the sums are added to
    the rows that tokens point to.  Returns dW."""
    yt = _type_code(dY, "dY")
    M, D = _two_dims(dY, "dY")
    dev = dY.get_device()
    tp, n, size = _tokens(tokens, dev)
    if n != M:
        raise ValueError(f"tokens has {n} elements, dY {M} rows")
    if dW is None:
        if V is None or accumulate:
            raise ValueError("dW is needed to accumulate" if accumulate else
                             "V, the rows of dW, is needed without dW")
    elif V is not None and V != _two_dims(dW, "dW")[0]:
        raise ValueError(f"dW has {dW.shape[0]} rows, V is {V}")
    else:
        V = _two_dims(dW, "dW")[0]
    y, ldy = _mat(dY, "dY", (dY.dtype,), M, D, dev)
    w, ldw = _mat(dW, "dW", _type_or_f32(dY.dtype), V, D, dev)
    _check_device(dev, "dY")
    if dW is None:
        dW, ldw = _new_rows(V, D, dY.dtype, dY, stream)
        w = dW.data_ptr()
    L = lib()
    need = L.embedding_backward_workspace_size(M, V, D)
    ws, nbytes = None, 0
    if need > 0:
        ws = _workspace(workspace, need, dY, stream)
        ws, nbytes = ws.data_ptr(), ws.numel()
    _check(L.embedding_backward(M, V, D, tp, size, y, ldy, yt, float(scale), int(bool(accumulate)),
                                w, ldw, _dtype_code(dW.dtype), ws, nbytes,
                                _handle(stream, dev)), "embedding_backward")
    return dW
