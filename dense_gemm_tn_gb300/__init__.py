"""Python binding of libdense_gemm_tn.so (the C ABI in include/tn_gemm.h).

Argument marshalling only: every step of the GEMM runs in the library's CUDA
kernels.  There is no CPU or PyTorch fallback -- importing this package
without the built library raises ImportError.

The same names as the C ABI:

    gemm_f16_tn(M, N, K, A, lda, B, ldb, C, ldc, stream=None)
    gemm_f8e4m3_tn(M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream=None)
    gemm_f8e4m3_tn_dscale(M, N, K, A, lda, B, ldb, C, ldc, scale_a_ptr, scale_b_ptr, stream=None)
    gemm_quantize_e4m3(x, x_type, rows, cols, ldx, q, ldq, scale_ptr, stream=None)
    gemm_f16_tn_softmax_stats(M, N, K, A, lda, B, ldb, C, ldc, scale, row_max, row_sum, stream=None)
    gemm_tn_grouped / gemm_tn_grouped_grad_b / gemm_tn_grouped_grad_a / gemm_i8_tn / gemm_i8_tn_grouped /
        gemm_quantize_i8_rows: products grouped by expert with their gradients, 8-bit integer products, row quantiser
    gemm_tn_gated / gemm_tn_gated_grad: gated projections act(gate) * up, dense and by expert, and their backward pass
    gemm_tn_cross_entropy / gemm_tn_cross_entropy_grad: softmax cross entropy of a projection onto a vocabulary
    gemm_w4_tn / gemm_quantize_w4_rows: products with 4-bit weights and group scales for few tokens, their quantiser
    gemm_poll_device_status(stream=None)

A, B and C are device pointers given as ints or as CUDA torch tensors (their
data_ptr() is passed; the tensor's shape is NOT consulted).

Two bindings of the same C functions: `lib` (ctypes) and, where build()
found the Python headers, `fast` (the CPython-API module _tn_fast, built from
csrc/pyfast.c: the same names and argument order, ints for pointers, about a
tenth of the per-call host time).  `calls` is `fast` when present, else
`lib`; the wrappers below go through it.  `stream` is an
int handle, a torch.cuda.Stream, or None for torch's current stream.  A
status other than GEMM_OK raises GemmError.

Convenience wrappers over torch tensors in TN storage:
    f16_tn(A (M,K) fp16, Bt (N,K) fp16, C=None) -> C^T as an (N, M) fp16 tensor
    f8e4m3_tn(A (M,K) uint8/float8_e4m3fn, Bt (N,K), scale_a, scale_b, C=None) -> (N, M) bf16
    tn_grouped(A (E,M,K), Bt (T,K), offsets (E+1,) int32, C=None) -> (T, M); tn_grouped_grad_b, tn_grouped_grad_a
    i8_tn(A (M,K) int8, Bt (N,K) int8, scale_a (M,), scale_b (N,), C=None) -> (N, M); i8_tn_grouped
    quantize_i8_rows(x (rows, cols)) -> (int8 codes, scale (rows,))
    tn_gated(A (2M,K) or (E,2M,K), Bt (T,K), offsets=None) -> (T, M); tn_gated_grad
    tn_cross_entropy(A (M,K), Bt (N,K), targets (N,) int64) -> (loss (N,), lse (N,)); tn_cross_entropy_grad
    w4_tn(A (M,ceil(K/2)) uint8, Bt (N,K), scale_a (M,groups), group) -> (N, M); quantize_w4_rows
The (N, M) row-major result IS the column-major M x N matrix C with ldc = M.
With a `stream`, new results are that stream's memory, as under torch.cuda.stream.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED = 2
GEMM_ERR_CUDA = 3
GEMM_ERR_TIMEOUT = 4

LIB_PATH = _build.LIB

#: C symbols the header declares (checked by the test suite).
EXPORTS = (
    "gemm_f16_tn", "gemm_f8e4m3_tn", "gemm_status_string", "gemm_last_error",
    "gemm_poll_device_status", "gemm_release_workspace", "gemm_tile_coord",
    "gemm_set_wait_limit_ns", "gemm_debug_inject_stall", "gemm_build_info",
    "gemm_f16_tn_noalloc", "gemm_debug_force_cta_group", "gemm_debug_force_wide_tiles", "gemm_debug_last_launch",
    "gemm_debug_set_raster_group", "gemm_debug_set_k_order", "gemm_debug_set_long_k_mode", "gemm_debug_set_lean_mode",
    "gemm_debug_set_skinny_mode",
    "gemm_debug_set_clock_probe",
    "gemm_f8e4m3_tn_dscale", "gemm_quantize_e4m3", "gemm_f16_tn_softmax_stats",
    "gemm_grouped_workspace", "gemm_tn_grouped", "gemm_tn_grouped_grad_b", "gemm_tn_grouped_grad_a",
    "gemm_i8_tn", "gemm_i8_tn_grouped", "gemm_quantize_i8_rows",
    "gemm_gated_workspace", "gemm_tn_gated", "gemm_tn_gated_grad",
    "gemm_cross_entropy_workspace", "gemm_tn_cross_entropy", "gemm_tn_cross_entropy_grad",
    "gemm_w4_tn", "gemm_quantize_w4_rows",
)

GEMM_IN_F32 = 0
GEMM_IN_F16 = 1
GEMM_IN_BF16 = 2

GEMM_GROUPED_PRODUCT = 0
GEMM_GROUPED_GRAD_B = 1
GEMM_GROUPED_GRAD_A = 2
GEMM_GROUPED_I8 = 3

GEMM_ACT_SILU = 0
GEMM_ACT_GELU = 1
GEMM_ACT_GELU_TANH = 2
#: Activations of tn_gated by name.
ACTIVATIONS = {"silu": GEMM_ACT_SILU, "gelu": GEMM_ACT_GELU, "gelu_tanh": GEMM_ACT_GELU_TANH}


class GemmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{status_string(status)}: {detail}" if detail else status_string(status))


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
            "(nvcc for sm_103a); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.gemm_f16_tn.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_f16_tn.restype = st
    lib.gemm_f8e4m3_tn.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64,
                                   ctypes.c_float, ctypes.c_float, vp]
    lib.gemm_f8e4m3_tn.restype = st
    lib.gemm_f8e4m3_tn_dscale.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp]
    lib.gemm_f8e4m3_tn_dscale.restype = st
    lib.gemm_f16_tn_softmax_stats.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, ctypes.c_float, vp, vp, vp]
    lib.gemm_f16_tn_softmax_stats.restype = st
    lib.gemm_quantize_e4m3.argtypes = [vp, st, i64, i64, i64, vp, i64, vp, vp]
    lib.gemm_quantize_e4m3.restype = st
    lib.gemm_f16_tn_noalloc.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_f16_tn_noalloc.restype = st
    lib.gemm_grouped_workspace.argtypes = [st, i64, i64, i64, i64, vp, i64, i64, vp, i64]
    lib.gemm_grouped_workspace.restype = i64
    lib.gemm_tn_grouped.argtypes = [st, i64, i64, i64, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp, i64, vp]
    lib.gemm_tn_grouped.restype = st
    lib.gemm_tn_grouped_grad_b.argtypes = [st, i64, i64, i64, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp, i64, vp]
    lib.gemm_tn_grouped_grad_b.restype = st
    lib.gemm_tn_grouped_grad_a.argtypes = [st, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, i64, vp, i64, vp]
    lib.gemm_tn_grouped_grad_a.restype = st
    lib.gemm_i8_tn.argtypes = [st, i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, i64, vp]
    lib.gemm_i8_tn.restype = st
    lib.gemm_i8_tn_grouped.argtypes = [st, i64, i64, i64, i64, vp, i64, i64, vp, vp, i64, vp, vp, vp, i64, vp, i64, vp]
    lib.gemm_i8_tn_grouped.restype = st
    lib.gemm_quantize_i8_rows.argtypes = [vp, st, i64, i64, i64, vp, i64, vp, vp]
    lib.gemm_quantize_i8_rows.restype = st
    lib.gemm_gated_workspace.argtypes = [st, st, i64, i64, i64, i64, vp, i64, i64, vp, i64]
    lib.gemm_gated_workspace.restype = i64
    lib.gemm_tn_gated.argtypes = [st, st, i64, i64, i64, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_tn_gated.restype = st
    lib.gemm_tn_gated_grad.argtypes = [st, st, i64, i64, i64, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64,
                                       vp, i64, vp, i64, vp]
    lib.gemm_tn_gated_grad.restype = st
    lib.gemm_cross_entropy_workspace.argtypes = [st, i64, i64, i64, vp, i64, vp, i64]
    lib.gemm_cross_entropy_workspace.restype = i64
    lib.gemm_tn_cross_entropy.argtypes = [st, i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp]
    lib.gemm_tn_cross_entropy.restype = st
    lib.gemm_tn_cross_entropy_grad.argtypes = [st, i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_tn_cross_entropy_grad.restype = st
    lib.gemm_w4_tn.argtypes = [st, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64, vp]
    lib.gemm_w4_tn.restype = st
    lib.gemm_quantize_w4_rows.argtypes = [vp, st, i64, i64, i64, i64, vp, i64, st, vp, i64, vp]
    lib.gemm_quantize_w4_rows.restype = st
    lib.gemm_status_string.argtypes = [st]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_last_error.argtypes = []
    lib.gemm_last_error.restype = ctypes.c_char_p
    lib.gemm_poll_device_status.argtypes = [vp]
    lib.gemm_poll_device_status.restype = st
    lib.gemm_release_workspace.argtypes = []
    lib.gemm_release_workspace.restype = None
    lib.gemm_tile_coord.argtypes = [i64, i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.gemm_tile_coord.restype = ctypes.c_int
    lib.gemm_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.gemm_set_wait_limit_ns.restype = None
    lib.gemm_debug_inject_stall.argtypes = [ctypes.c_int]
    lib.gemm_debug_inject_stall.restype = None
    lib.gemm_debug_force_cta_group.argtypes = [ctypes.c_int]
    lib.gemm_debug_force_cta_group.restype = ctypes.c_int
    lib.gemm_debug_force_wide_tiles.argtypes = [ctypes.c_int]
    lib.gemm_debug_force_wide_tiles.restype = ctypes.c_int
    lib.gemm_debug_set_raster_group.argtypes = [ctypes.c_int]
    lib.gemm_debug_set_raster_group.restype = ctypes.c_int
    lib.gemm_debug_set_clock_probe.argtypes = [ctypes.c_void_p]
    lib.gemm_debug_set_clock_probe.restype = None
    lib.gemm_debug_set_long_k_mode.argtypes = [ctypes.c_int]
    lib.gemm_debug_set_long_k_mode.restype = ctypes.c_int
    lib.gemm_debug_set_lean_mode.argtypes = [ctypes.c_int]
    lib.gemm_debug_set_lean_mode.restype = ctypes.c_int
    lib.gemm_debug_set_skinny_mode.argtypes = [ctypes.c_int]
    lib.gemm_debug_set_skinny_mode.restype = ctypes.c_int
    lib.gemm_debug_set_k_order.argtypes = [ctypes.c_int]
    lib.gemm_debug_set_k_order.restype = ctypes.c_int
    lib.gemm_debug_last_launch.argtypes = []
    lib.gemm_debug_last_launch.restype = ctypes.c_char_p
    lib.gemm_build_info.argtypes = []
    lib.gemm_build_info.restype = ctypes.c_char_p
    return lib


_lib = _load()
lib = _lib

try:
    # loads after _lib: it links the same library file, which the dynamic
    # loader then shares with the ctypes binding (one device state)
    from . import _tn_fast as fast
except ImportError:
    fast = None
calls = fast if fast is not None else _lib


def status_string(status: int) -> str:
    return _lib.gemm_status_string(int(status)).decode()


def last_error() -> str:
    return _lib.gemm_last_error().decode()


def last_launch() -> str:
    return _lib.gemm_debug_last_launch().decode()


def build_info() -> str:
    return _lib.gemm_build_info().decode()


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int) -> int:
    if status != GEMM_OK:
        detail = last_error()
        if status == GEMM_ERR_CUDA and last_launch():
            detail += f" (last launch: {last_launch()})"
        raise GemmError(status, detail)
    return status


def gemm_f16_tn(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return _check(calls.gemm_f16_tn(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _stream(stream)))


def gemm_f8e4m3_tn(M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream=None) -> int:
    return _check(calls.gemm_f8e4m3_tn(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                       float(scale_a), float(scale_b), _stream(stream)))


def gemm_f8e4m3_tn_dscale(M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream=None) -> int:
    """gemm_f8e4m3_tn with scale_a / scale_b as device pointers (one fp32 each)."""
    return _check(calls.gemm_f8e4m3_tn_dscale(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                              _ptr(scale_a), _ptr(scale_b), _stream(stream)))


def gemm_f16_tn_softmax_stats(M, N, K, A, lda, B, ldb, C, ldc, scale, row_max, row_sum, stream=None) -> int:
    """Scaled scores C = fp16(scale * A B) with the softmax row statistics
    (row_max, row_sum: device float arrays of M)."""
    return _check(calls.gemm_f16_tn_softmax_stats(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, float(scale),
                                                  _ptr(row_max), _ptr(row_sum), _stream(stream)))


def gemm_quantize_e4m3(x, x_type, rows, cols, ldx, q, ldq, scale, stream=None) -> int:
    """Per-tensor E4M3 quantisation on the device: codes into q, amax / 448 into *scale."""
    return _check(calls.gemm_quantize_e4m3(_ptr(x), int(x_type), rows, cols, ldx, _ptr(q), ldq, _ptr(scale),
                                           _stream(stream)))


def gemm_grouped_workspace(op, E, M, K, T, X, ldx, stride_x, Y, ldy) -> int:
    """Workspace bytes that a grouped or 8-bit product with these operands needs."""
    n = calls.gemm_grouped_workspace(int(op), E, M, K, T, _ptr(X), ldx, stride_x, _ptr(Y), ldy)
    if n < 0:
        raise ValueError("gemm_grouped_workspace: argument out of range")
    return n


def gemm_tn_grouped(type, E, M, K, T, A, lda, stride_a, B, ldb, offsets, C, ldc, workspace=None, workspace_bytes=0,
                    stream=None) -> int:
    return _check(calls.gemm_tn_grouped(int(type), E, M, K, T, _ptr(A), lda, stride_a, _ptr(B), ldb, _ptr(offsets),
                                        _ptr(C), ldc, _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_tn_grouped_grad_b(type, E, M, K, T, A, lda, stride_a, dC, lddc, offsets, dB, lddb, workspace=None,
                           workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_tn_grouped_grad_b(int(type), E, M, K, T, _ptr(A), lda, stride_a, _ptr(dC), lddc,
                                               _ptr(offsets), _ptr(dB), lddb, _ptr(workspace), workspace_bytes,
                                               _stream(stream)))


def gemm_tn_grouped_grad_a(type, E, M, K, T, dC, lddc, B, ldb, offsets, dA, ldda, stride_da, workspace=None,
                           workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_tn_grouped_grad_a(int(type), E, M, K, T, _ptr(dC), lddc, _ptr(B), ldb, _ptr(offsets),
                                               _ptr(dA), ldda, stride_da, _ptr(workspace), workspace_bytes,
                                               _stream(stream)))


def gemm_i8_tn(out_type, M, N, K, A, lda, scale_a, B, ldb, scale_b, C, ldc, workspace=None, workspace_bytes=0,
               stream=None) -> int:
    return _check(calls.gemm_i8_tn(int(out_type), M, N, K, _ptr(A), lda, _ptr(scale_a), _ptr(B), ldb, _ptr(scale_b),
                                   _ptr(C), ldc, _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_i8_tn_grouped(out_type, E, M, K, T, A, lda, stride_a, scale_a, B, ldb, scale_b, offsets, C, ldc,
                       workspace=None, workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_i8_tn_grouped(int(out_type), E, M, K, T, _ptr(A), lda, stride_a, _ptr(scale_a), _ptr(B),
                                           ldb, _ptr(scale_b), _ptr(offsets), _ptr(C), ldc, _ptr(workspace),
                                           workspace_bytes, _stream(stream)))


def gemm_quantize_i8_rows(x, x_type, rows, cols, ldx, q, ldq, scale, stream=None) -> int:
    """8-bit quantisation with a scale per row: codes into q, amax / 127 of each row into scale."""
    return _check(calls.gemm_quantize_i8_rows(_ptr(x), int(x_type), rows, cols, ldx, _ptr(q), ldq, _ptr(scale),
                                              _stream(stream)))


def gemm_gated_workspace(grad, dense, E, M, K, T, A, lda, stride_a, B, ldb) -> int:
    """Workspace bytes of gemm_tn_gated (grad 0) or gemm_tn_gated_grad (grad 1); dense: without offsets."""
    n = calls.gemm_gated_workspace(int(grad), int(dense), E, M, K, T, _ptr(A), lda, stride_a, _ptr(B), ldb)
    if n < 0:
        raise ValueError("gemm_gated_workspace: argument out of range")
    return n


def gemm_tn_gated(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, H, ldh, P=None, ldp=0, workspace=None,
                  workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_tn_gated(int(type), int(act), E, M, K, T, _ptr(A), lda, stride_a, _ptr(B), ldb, _ptr(offsets),
                                      _ptr(H), ldh, _ptr(P), ldp, _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_tn_gated_grad(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, P, ldp, dH, lddh, dA, ldda, stride_da, dB,
                       lddb, workspace=None, workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_tn_gated_grad(int(type), int(act), E, M, K, T, _ptr(A), lda, stride_a, _ptr(B), ldb,
                                           _ptr(offsets), _ptr(P), ldp, _ptr(dH), lddh, _ptr(dA), ldda, stride_da, _ptr(dB),
                                           lddb, _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_cross_entropy_workspace(grad, M, N, K, A, lda, B, ldb) -> int:
    """Workspace bytes of gemm_tn_cross_entropy (grad 0) or gemm_tn_cross_entropy_grad (grad 1)."""
    n = calls.gemm_cross_entropy_workspace(int(grad), M, N, K, _ptr(A), lda, _ptr(B), ldb)
    if n < 0:
        raise ValueError("gemm_cross_entropy_workspace: argument out of range")
    return n


def gemm_tn_cross_entropy(type, M, N, K, A, lda, B, ldb, targets, loss, lse, workspace=None, workspace_bytes=0,
                          stream=None) -> int:
    return _check(calls.gemm_tn_cross_entropy(int(type), M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(targets), _ptr(loss),
                                              _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_tn_cross_entropy_grad(type, M, N, K, A, lda, B, ldb, targets, lse, dloss, dA, ldda, dB, lddb, workspace=None,
                               workspace_bytes=0, stream=None) -> int:
    return _check(calls.gemm_tn_cross_entropy_grad(int(type), M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(targets), _ptr(lse),
                                                   _ptr(dloss), _ptr(dA), ldda, _ptr(dB), lddb, _ptr(workspace),
                                                   workspace_bytes, _stream(stream)))


def gemm_w4_tn(type, M, N, K, A, lda, scale_a, ld_scale, group, B, ldb, C, ldc, stream=None) -> int:
    return _check(calls.gemm_w4_tn(int(type), M, N, K, _ptr(A), lda, _ptr(scale_a), ld_scale, group, _ptr(B), ldb, _ptr(C),
                                   ldc, _stream(stream)))


def gemm_quantize_w4_rows(x, x_type, rows, cols, ldx, group, q, ldq, scale_type, scale, ld_scale, stream=None) -> int:
    """4-bit quantisation with a scale per group of a row's terms: two codes a byte into q."""
    return _check(calls.gemm_quantize_w4_rows(_ptr(x), int(x_type), rows, cols, ldx, group, _ptr(q), ldq, int(scale_type),
                                              _ptr(scale), ld_scale, _stream(stream)))


def gemm_f16_tn_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    """gemm_f16_tn for callers that cannot let the library allocate device
    memory (their own memory pool or budget, or no implicit synchronisation
    allowed): operand copies go to a fixed 32 MiB array in the library's
    device image instead of a cudaMalloc'd workspace."""
    return _check(calls.gemm_f16_tn_noalloc(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                            _stream(stream)))


def gemm_poll_device_status(stream=None) -> int:
    return _check(_lib.gemm_poll_device_status(_stream(stream)))


def gemm_release_workspace() -> None:
    _lib.gemm_release_workspace()


def gemm_tile_coord(tiles_m, tiles_n, group, tile_id):
    tm, tn = ctypes.c_int64(), ctypes.c_int64()
    rc = _lib.gemm_tile_coord(tiles_m, tiles_n, group, tile_id, ctypes.byref(tm), ctypes.byref(tn))
    if rc != 0:
        raise ValueError("gemm_tile_coord: argument out of range")
    return tm.value, tn.value


def gemm_set_wait_limit_ns(limit_ns: int) -> None:
    _lib.gemm_set_wait_limit_ns(int(limit_ns))


def gemm_debug_inject_stall(mode) -> None:
    """0 off; 1 stall the MMA thread; 2 / 3 stall the even / odd CTA's producer."""
    _lib.gemm_debug_inject_stall(int(mode))


def gemm_debug_force_cta_group(group: int) -> None:
    if _lib.gemm_debug_force_cta_group(int(group)) != 0:
        raise ValueError("cta group must be 0 (automatic), 1 or 2")


def gemm_debug_force_wide_tiles(mode: int) -> None:
    """0 automatic; 1 CTA pairs always compute 256 x 512 tiles; -1 never."""
    if _lib.gemm_debug_force_wide_tiles(int(mode)) != 0:
        raise ValueError("mode must be -1, 0 or 1")


def gemm_debug_set_raster_group(rows: int) -> None:
    """Tile rows per raster group of the scheduler (even, 2 .. 64); 0 the default."""
    if _lib.gemm_debug_set_raster_group(int(rows)) != 0:
        raise ValueError("rows must be 0 or an even number up to 64")


def gemm_debug_set_k_order(mode: int) -> None:
    """0 the library's choice; 1 every tile walks K forward; 2 odd waves walk it backwards."""
    if _lib.gemm_debug_set_k_order(int(mode)) != 0:
        raise ValueError("mode must be 0, 1 or 2")


def gemm_debug_set_clock_probe(counters) -> None:
    """A device pointer (int) to 3 zeroed 64-bit words, or None: while set,
    each GEMM launch adds its SM cycles, nanoseconds and 1 to them."""
    _lib.gemm_debug_set_clock_probe(None if counters is None else ctypes.c_void_p(int(counters)))


def gemm_debug_set_long_k_mode(mode: int) -> None:
    """0 the library's choice; 1 split-reduce (HBM partials); 2 reduce inside a cluster of single CTAs."""
    if _lib.gemm_debug_set_long_k_mode(int(mode)) != 0:
        raise ValueError("mode must be 0, 1 or 2")


def gemm_debug_set_skinny_mode(mode: int) -> None:
    """N <= 64: 0 the library's choice; 1 never the skinny kernel; 2 always."""
    if _lib.gemm_debug_set_skinny_mode(int(mode)) != 0:
        raise ValueError("mode must be 0, 1 or 2")


def gemm_debug_set_lean_mode(mode: int) -> None:
    """m-part launches: 0 the library's choice; 1 the full configuration; 2 the
    lean one (two CTAs per SM) wherever the units are quarters or halves."""
    if _lib.gemm_debug_set_lean_mode(int(mode)) != 0:
        raise ValueError("mode must be 0, 1 or 2")


# ---------------------------------------------------------------- torch helpers
def _rows(t, dtype, name, shape=None, cuda=True):
    """Checks a 2-D CUDA tensor of `dtype` whose rows are contiguous (the layout
    the C ABI reads with a leading dimension) and returns its row stride."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its second dimension")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _operands(A, Bt, dtype):
    """(M, N, K, lda, ldb) of A (M, K) and Bt (N, K), both checked by _rows."""
    lda = _rows(A, dtype, "A", cuda=False)
    ldb = _rows(Bt, dtype, "Bt", cuda=False)
    (M, K), N = A.shape, Bt.shape[0]
    if Bt.shape[1] != K:
        raise ValueError(f"A is {tuple(A.shape)} and Bt {tuple(Bt.shape)}: their second dimensions (K) differ")
    for t, name in ((A, "A"), (Bt, "Bt")):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    if A.device != Bt.device:
        raise ValueError("A and Bt must be on the same device")
    return M, N, K, lda, ldb


def _torch_stream(device, stream):
    """The torch stream of a `stream` argument (not None).  Handle 0 is the default
    stream: torch.cuda.ExternalStream would make it one of torch's pool."""
    import torch
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, stream):
    """A result's tensor.  On a stream of the caller's its memory is that stream's, as
    under torch.cuda.stream(stream): the current stream may still have kernels in hand
    that use what its own freed blocks held.  Once released it waits for the current
    stream as well, whose kernels may read the result."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(device, stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _output(C, M, N, dtype, device, stream=None):
    if C is None:
        C = _empty((N, M), dtype, device, stream)
    ldc = _rows(C, dtype, "C", (N, M))
    if C.device != device:
        raise ValueError(f"C is on {C.device}, the operands on {device}")
    return C, ldc


def _on(device):
    """The C ABI works on the calling thread's current device: make it the
    operands' device for the call."""
    import torch
    return torch.cuda.device(device)


def f16_tn(A, Bt, C=None, stream=None):
    """C^T (N, M) = Bt (N, K) @ A (M, K)^T, i.e. column-major C = A x B.
    A, Bt (and C) are fp16 CUDA tensors whose rows are contiguous."""
    import torch
    M, N, K, lda, ldb = _operands(A, Bt, torch.float16)
    C, ldc = _output(C, M, N, torch.float16, A.device, stream)
    with _on(A.device):
        gemm_f16_tn(M, N, K, A, lda, Bt, ldb, C, ldc, stream)
    return C


def f16_tn_softmax_stats(Q, Kmat, scale, C=None, stream=None):
    """Q (M, K) and Kmat (N, K) fp16 CUDA tensors -> (S^T as an (N, M) fp16
    tensor, row_max (M,), row_sum (M,)): S = scale * Q Kmat^T."""
    import torch
    M, N, K, lda, ldb = _operands(Q, Kmat, torch.float16)
    C, ldc = _output(C, M, N, torch.float16, Q.device, stream)
    row_max, row_sum = (_empty((M,), torch.float32, Q.device, stream) for _ in range(2))
    with _on(Q.device):
        gemm_f16_tn_softmax_stats(M, N, K, Q, lda, Kmat, ldb, C, ldc, scale, row_max, row_sum, stream)
    return C, row_max, row_sum


def quantize_e4m3(x, stream=None):
    """x: a 2-D float32 / float16 / bfloat16 CUDA tensor with unit column
    stride.  Returns (codes as a uint8 tensor of x's shape, scale as a
    1-element float32 tensor), both on x's device."""
    import torch
    types = {torch.float32: GEMM_IN_F32, torch.float16: GEMM_IN_F16, torch.bfloat16: GEMM_IN_BF16}
    if x.dtype not in types or x.dim() != 2 or (x.numel() > 0 and x.stride(1) != 1):
        raise ValueError("x must be a 2-D float32/float16/bfloat16 tensor with unit column stride")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    rows, cols = x.shape
    q = _empty((rows, cols), torch.uint8, x.device, stream)
    scale = _empty((1,), torch.float32, x.device, stream)
    ld = max(cols, 1)
    with _on(x.device):
        gemm_quantize_e4m3(x, types[x.dtype], rows, cols, x.stride(0) if rows > 1 else ld, q, ld, scale, stream)
    return q, scale


def _scale_tensor(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda or t.numel() < 1:
        raise ValueError(f"{name} must be a float32 CUDA tensor with at least one element")


def f8e4m3_tn_dscale(A, Bt, scale_a, scale_b, C=None, stream=None):
    """f8e4m3_tn with the scales as 1-element float32 CUDA tensors.  A, Bt:
    uint8 E4M3 codes (CUDA, rows contiguous); C: bf16 (N, M)."""
    import torch
    M, N, K, lda, ldb = _operands(A, Bt, torch.uint8)
    _scale_tensor(scale_a, "scale_a")
    _scale_tensor(scale_b, "scale_b")
    if scale_a.device != A.device or scale_b.device != A.device:
        raise ValueError("scale_a and scale_b must be on the operands' device")
    C, ldc = _output(C, M, N, torch.bfloat16, A.device, stream)
    with _on(A.device):
        gemm_f8e4m3_tn_dscale(M, N, K, A, lda, Bt, ldb, C, ldc, scale_a, scale_b, stream)
    return C


def f8e4m3_tn(A, Bt, scale_a, scale_b, C=None, stream=None):
    """C^T (N, M) = bf16(scale_a * scale_b * Bt A^T) for uint8 E4M3 codes A
    (M, K) and Bt (N, K); the scales are Python floats."""
    import torch
    M, N, K, lda, ldb = _operands(A, Bt, torch.uint8)
    C, ldc = _output(C, M, N, torch.bfloat16, A.device, stream)
    with _on(A.device):
        gemm_f8e4m3_tn(M, N, K, A, lda, Bt, ldb, C, ldc, float(scale_a), float(scale_b), stream)
    return C


# ---------------------------------------------------------------- grouped and 8-bit products
# Each helper checks its arguments in full, except that operands which are all
# contiguous on the current device (the common case, and the one where a call is
# short enough for the host's time to count) take a shorter way through the same
# checks of types and shapes.  Measured on a GB300's host (a plain torch.add takes 7.9 us
# there): tn_grouped_grad_a 24.9 -> 14.1 us a call.
_torch = None          # the module, from the first helper call on
_half_kinds = {}       # {dtype: GEMM_IN_...} of the 16-bit types


def _load_torch():
    global _torch
    import torch
    _half_kinds.update({torch.float16: GEMM_IN_F16, torch.bfloat16: GEMM_IN_BF16})
    _torch = torch
    return torch


def _half_type(dtype, name):
    kind = _half_kinds.get(dtype)
    if kind is not None:
        return kind
    raise ValueError(f"{name} must be torch.float16 or torch.bfloat16, not {dtype}")


def _experts(t, dtype, name, shape=None):
    """(row stride, expert stride) of a 3-D tensor (E, rows, inner) with contiguous rows."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D torch tensor (experts, rows, columns)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    E, R, I = t.shape
    if shape is not None and (E, R, I) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {(E, R, I)}")
    s0, s1, s2 = t.stride()
    if I > 1 and s2 != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return (s1 if R > 1 else max(I, 1)), (s0 if E > 1 else 0)


def _vector(t, dtype, n, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},)")


def _tokens(t, dtype, cols, name):
    """Row stride of a 2-D tensor of `cols` columns (rows contiguous)."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name} must be a 2-D torch tensor with {cols} columns")
    return _rows(t, dtype, name, cuda=False)


def _same_device(device, **tensors):
    if device.type != "cuda":
        raise ValueError("the tensors must be CUDA tensors")
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _launch_stream(index, stream):
    """The stream's handle (None: torch's current stream of that device)."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _workspace(device, stream, n):
    """n bytes from torch's allocator that belong to the call's stream, so that
    they are used again only after the call's kernels."""
    torch = _torch
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_torch_stream(device, stream)):
        return torch.empty(n, dtype=torch.uint8, device=device)


#: Bytes that a workspace with tensor maps goes on for behind what the call needs.  A call whose maps lay in the last
#: 53 KiB before unmapped memory failed with an illegal address on a GB300, twice in the same place, and no access of the
#: kernels leads there; with the same maps further from the end it never has.
_BEHIND_MAPS = 1 << 16


def _tensors(torch, *operands):
    for t in operands:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"the operands must be torch tensors, not {type(t).__name__}")


def _plain(torch, *tensors):
    """Whether the tensors are contiguous on the current device: their strides are
    their shapes', and nothing is left to check but types and shapes."""
    index = tensors[0].get_device()
    for t in tensors:
        if not t.is_contiguous() or t.get_device() != index:
            return False
    return index >= 0 and torch._C._cuda_getDevice() == index


def _elsewhere(index):
    """Whether device `index` is not the calling thread's current one (which the C ABI works on)."""
    return _torch._C._cuda_getDevice() != index


def tn_grouped(A, Bt, offsets, C=None, stream=None):
    """C^T[t] = A[e] Bt[t] for the rows offsets[e] <= t < offsets[e + 1] of every
    expert e: A (E, M, K), Bt (T, K), offsets (E + 1,) int32, all on one GPU;
    A, Bt and C (T, M) are all fp16 or all bf16, their rows contiguous.  Rows of
    no expert are not written."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, offsets)
    dtype, device, sa, sb, so = A.dtype, A.device, A.shape, Bt.shape, offsets.shape
    kind = _half_type(dtype, "A")
    if (C is None and Bt.dtype is dtype and offsets.dtype is torch.int32 and len(sa) == 3 and len(sb) == 2
            and len(so) == 1 and sa[2] == sb[1] > 0 and so[0] == sa[0] + 1 and _plain(torch, A, Bt, offsets)):
        (E, M, K), T = sa, sb[0]
        lda = ldb = K
        stride_a = M * K
        C, ldc = _empty((T, M), dtype, device, stream), max(M, 1)
    else:
        lda, stride_a = _experts(A, dtype, "A")
        E, M, K = A.shape
        ldb, T = _tokens(Bt, dtype, K, "Bt"), Bt.shape[0]
        _vector(offsets, torch.int32, E + 1, "offsets")
        _same_device(device, Bt=Bt, offsets=offsets)
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return tn_grouped(A, Bt, offsets, C, stream)
        C, ldc = _output(C, M, T, dtype, device, stream)
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_grouped_workspace(GEMM_GROUPED_PRODUCT, E, M, K, T, a, lda, stride_a, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    ws = held.data_ptr() if n > 0 else None
    _check(calls.gemm_tn_grouped(kind, E, M, K, T, a, lda, stride_a, b, ldb, offsets.data_ptr(), C.data_ptr(), ldc, ws,
                                 n, _launch_stream(device.index, stream)))
    return C


def tn_grouped_grad_b(A, dCt, offsets, dBt=None, stream=None):
    """The gradient of tn_grouped for Bt: dBt[t] = A[e]^T dC^T[t], with dCt (T, M)
    -> (T, K).  Rows of no expert are not written."""
    torch = _torch or _load_torch()
    _tensors(torch, A, dCt, offsets)
    dtype, device, sa, sd, so = A.dtype, A.device, A.shape, dCt.shape, offsets.shape
    kind = _half_type(dtype, "A")
    if (dBt is None and dCt.dtype is dtype and offsets.dtype is torch.int32 and len(sa) == 3 and len(sd) == 2
            and len(so) == 1 and sa[1] == sd[1] > 0 < sa[2] and so[0] == sa[0] + 1 and _plain(torch, A, dCt, offsets)):
        (E, M, K), T = sa, sd[0]
        lda, stride_a, ldd = K, M * K, M
        dBt, ldb = _empty((T, K), dtype, device, stream), K
    else:
        lda, stride_a = _experts(A, dtype, "A")
        E, M, K = A.shape
        ldd, T = _tokens(dCt, dtype, M, "dCt"), dCt.shape[0]
        _vector(offsets, torch.int32, E + 1, "offsets")
        _same_device(device, dCt=dCt, offsets=offsets)
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return tn_grouped_grad_b(A, dCt, offsets, dBt, stream)
        dBt, ldb = _output(dBt, K, T, dtype, device, stream)
    a, d = A.data_ptr(), dCt.data_ptr()
    n = calls.gemm_grouped_workspace(GEMM_GROUPED_GRAD_B, E, M, K, T, a, lda, stride_a, d, ldd)
    held = _workspace(device, stream, n) if n > 0 else None
    ws = held.data_ptr() if n > 0 else None
    _check(calls.gemm_tn_grouped_grad_b(kind, E, M, K, T, a, lda, stride_a, d, ldd, offsets.data_ptr(), dBt.data_ptr(),
                                        ldb, ws, n, _launch_stream(device.index, stream)))
    return dBt


def tn_grouped_grad_a(dCt, Bt, offsets, dA=None, stream=None):
    """The gradient of tn_grouped for A: dA[e] = sum over e's rows t of the outer
    products dC^T[t] Bt[t], with dCt (T, M) and Bt (T, K) -> (E, M, K); zeros for
    an expert without rows."""
    torch = _torch or _load_torch()
    _tensors(torch, dCt, Bt, offsets)
    dtype, device, sd, sb, so = dCt.dtype, dCt.device, dCt.shape, Bt.shape, offsets.shape
    if len(so) != 1 or so[0] < 1:
        raise ValueError("offsets must be a 1-D tensor of experts + 1 row numbers")
    if len(sd) != 2 or len(sb) != 2:
        raise ValueError("dCt and Bt must be 2-D torch tensors")
    E, (T, M), K = so[0] - 1, sd, sb[1]
    kind = _half_type(dtype, "dCt")
    if (dA is None and Bt.dtype is dtype and offsets.dtype is torch.int32 and sb[0] == T and M > 0 < K
            and _plain(torch, dCt, Bt, offsets)):
        ldd, ldb, ldda, stride_da = M, K, K, M * K
        dA = _empty((E, M, K), dtype, device, stream)
    else:
        ldd, ldb = _tokens(dCt, dtype, M, "dCt"), _tokens(Bt, dtype, K, "Bt")
        if sb[0] != T:
            raise ValueError(f"dCt has {T} rows and Bt {sb[0]}")
        _vector(offsets, torch.int32, E + 1, "offsets")
        _same_device(device, Bt=Bt, offsets=offsets)
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return tn_grouped_grad_a(dCt, Bt, offsets, dA, stream)
        if dA is None:
            dA = _empty((E, M, K), dtype, device, stream)
        ldda, stride_da = _experts(dA, dtype, "dA", (E, M, K))
        _same_device(device, dA=dA)
    d, b = dCt.data_ptr(), Bt.data_ptr()
    n = calls.gemm_grouped_workspace(GEMM_GROUPED_GRAD_A, E, M, K, T, d, ldd, 0, b, ldb)
    held = _workspace(device, stream, n + _BEHIND_MAPS) if n > 0 else None
    ws = held.data_ptr() if n > 0 else None
    _check(calls.gemm_tn_grouped_grad_a(kind, E, M, K, T, d, ldd, b, ldb, offsets.data_ptr(), dA.data_ptr(), ldda,
                                        stride_da, ws, n, _launch_stream(device.index, stream)))
    return dA


def i8_tn(A, Bt, scale_a, scale_b, C=None, dtype=None, stream=None):
    """C^T[n, m] = scale_a[m] scale_b[n] sum_k A[m, k] Bt[n, k]: A (M, K) and Bt
    (N, K) int8, scale_a (M,) and scale_b (N,) fp32 -> (N, M) of `dtype`
    (torch.float16, unless C or dtype says torch.bfloat16)."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, scale_a, scale_b)
    dtype, device, sa, sb = dtype or (torch.float16 if C is None else C.dtype), A.device, A.shape, Bt.shape
    kind = _half_type(dtype, "dtype")
    if (C is None and A.dtype is torch.int8 is Bt.dtype and scale_a.dtype is torch.float32 is scale_b.dtype
            and len(sa) == 2 == len(sb) and sa[1] == sb[1] > 0 and scale_a.shape == (sa[0],) and scale_b.shape == (sb[0],)
            and _plain(torch, A, Bt, scale_a, scale_b)):
        (M, K), N = sa, sb[0]
        lda = ldb = K
        C, ldc = _empty((N, M), dtype, device, stream), max(M, 1)
    else:
        M, N, K, lda, ldb = _operands(A, Bt, torch.int8)
        _vector(scale_a, torch.float32, M, "scale_a")
        _vector(scale_b, torch.float32, N, "scale_b")
        _same_device(device, scale_a=scale_a, scale_b=scale_b)
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return i8_tn(A, Bt, scale_a, scale_b, C, dtype, stream)
        C, ldc = _output(C, M, N, dtype, device, stream)
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_grouped_workspace(GEMM_GROUPED_I8, 1, M, K, N, a, lda, 0, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    ws = held.data_ptr() if n > 0 else None
    _check(calls.gemm_i8_tn(kind, M, N, K, a, lda, scale_a.data_ptr(), b, ldb, scale_b.data_ptr(), C.data_ptr(), ldc, ws,
                            n, _launch_stream(device.index, stream)))
    return C


def _i8_grouped_operands(A, Bt, scale_a, scale_b, offsets, C, dtype, stream):
    """(lda, stride_a, ldb, ldc, C) of i8_tn_grouped's operands, all checked."""
    import torch
    lda, stride_a = _experts(A, torch.int8, "A")
    E, M, K = A.shape
    ldb, T = _tokens(Bt, torch.int8, K, "Bt"), Bt.shape[0]
    if (not isinstance(scale_a, torch.Tensor) or scale_a.dtype != torch.float32 or tuple(scale_a.shape) != (E, M)
            or not scale_a.is_contiguous()):
        raise ValueError(f"scale_a must be a contiguous torch.float32 tensor of shape {(E, M)}")
    _vector(scale_b, torch.float32, T, "scale_b")
    _vector(offsets, torch.int32, E + 1, "offsets")
    _same_device(A.device, Bt=Bt, scale_a=scale_a, scale_b=scale_b, offsets=offsets)
    C, ldc = _output(C, M, T, dtype, A.device, stream)
    return lda, stride_a, ldb, ldc, C


def i8_tn_grouped(A, Bt, scale_a, scale_b, offsets, C=None, dtype=None, stream=None):
    """i8_tn grouped by expert as in tn_grouped: A (E, M, K) and Bt (T, K) int8,
    scale_a (E, M) and scale_b (T,) fp32 -> (T, M) of `dtype`."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, scale_a, scale_b, offsets)
    dtype, device, sa, sb = dtype or (torch.float16 if C is None else C.dtype), A.device, A.shape, Bt.shape
    kind = _half_type(dtype, "dtype")
    if (C is None and A.dtype is torch.int8 is Bt.dtype and scale_a.dtype is torch.float32 is scale_b.dtype
            and offsets.dtype is torch.int32 and len(sa) == 3 and len(sb) == 2 and sa[2] == sb[1] > 0 < sa[1]
            and scale_a.shape == sa[:2] and scale_b.shape == (sb[0],) and offsets.shape == (sa[0] + 1,)
            and _plain(torch, A, Bt, scale_a, scale_b, offsets)):
        (E, M, K), T = sa, sb[0]
        lda = ldb = K
        stride_a = M * K
        C, ldc = _empty((T, M), dtype, device, stream), M
    else:
        lda, stride_a, ldb, ldc, C = _i8_grouped_operands(A, Bt, scale_a, scale_b, offsets, C, dtype, stream)
        (E, M, K), T = A.shape, Bt.shape[0]
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return i8_tn_grouped(A, Bt, scale_a, scale_b, offsets, C, dtype, stream)
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_grouped_workspace(GEMM_GROUPED_I8, E, M, K, T, a, lda, stride_a, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    ws = held.data_ptr() if n > 0 else None
    _check(calls.gemm_i8_tn_grouped(kind, E, M, K, T, a, lda, stride_a, scale_a.data_ptr(), b, ldb, scale_b.data_ptr(),
                                    offsets.data_ptr(), C.data_ptr(), ldc, ws, n, _launch_stream(device.index, stream)))
    return C


def quantize_i8_rows(x, stream=None):
    """x: a 2-D float32 / float16 / bfloat16 CUDA tensor with unit column stride.
    Returns (int8 codes of x's shape, scale as a float32 tensor of its rows): the
    operands of i8_tn, for activations (tokens) and weights (channels) alike."""
    torch = _torch or _load_torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D float32/float16/bfloat16 tensor")
    dtype, device = x.dtype, x.device
    kind = GEMM_IN_F32 if dtype is torch.float32 else _half_kinds.get(dtype)
    if kind is None:
        raise ValueError("x must be a 2-D float32/float16/bfloat16 tensor")
    shape = x.shape
    rows, cols = shape
    if cols > 0 and _plain(torch, x):
        ldx = cols
    else:
        ldx = _rows(x, dtype, "x")
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return quantize_i8_rows(x, stream)
    q = _empty(shape, torch.int8, device, stream)
    scale = _empty((rows,), torch.float32, device, stream)
    _check(calls.gemm_quantize_i8_rows(x.data_ptr(), kind, rows, cols, ldx, q.data_ptr(), max(cols, 1), scale.data_ptr(),
                                       _launch_stream(device.index, stream)))
    return q, scale


# ---------------------------------------------------------------- gated projections and the vocabulary's loss
def _gated_operands(A, Bt, offsets, P=None, dHt=None):
    """(E, M, K, T, lda, stride_a, ldb, ldp, lddh) of gate and up rows A, (E, 2 M, K) with offsets and (2 M, K)
    without, of tokens Bt (T, K) and, for the gradient, of products P (T, 2 M) and gradients dHt (T, M)."""
    torch, dtype, sa, sb = _torch, A.dtype, A.shape, Bt.shape
    if (len(sa) == (2 if offsets is None else 3) and len(sb) == 2 and sa[-1] == sb[1] > 0 and sa[-2] % 2 == 0 < sa[-2]
            and Bt.dtype is dtype and _plain(torch, A, Bt)):
        T, K, rows, E = sb[0], sb[1], sa[-2], 1 if offsets is None else sa[0]
        M = rows // 2
        if ((offsets is None or (isinstance(offsets, torch.Tensor) and offsets.dtype is torch.int32
                                 and offsets.shape == (E + 1,) and _plain(torch, offsets)))
                and (P is None or (P.dtype is torch.float32 and P.shape == (T, rows) and dHt.dtype is dtype
                                   and dHt.shape == (T, M) and _plain(torch, P, dHt)))):
            return E, M, K, T, K, (rows * K if E > 1 else 0), K, rows, M
    stride_a = ldp = lddh = 0
    if offsets is None:
        lda = _rows(A, dtype, "A", cuda=False)
        E, (rows, K) = 1, A.shape
    else:
        lda, stride_a = _experts(A, dtype, "A")
        E, rows, K = A.shape
        _vector(offsets, torch.int32, E + 1, "offsets")
    if rows % 2:
        raise ValueError(f"A must have an even number of rows (gate rows, then up rows), not {rows}")
    ldb, T, M = _tokens(Bt, dtype, K, "Bt"), Bt.shape[0], rows // 2
    if P is not None:
        ldp = _rows(P, torch.float32, "P", (T, rows), cuda=False)
    if dHt is not None:
        lddh = _rows(dHt, dtype, "dHt", (T, M), cuda=False)
    others = {"Bt": Bt, "P": P, "dHt": dHt, "offsets": offsets}
    _same_device(A.device, **{name: t for name, t in others.items() if t is not None})
    return E, M, K, T, lda, stride_a, ldb, ldp, lddh


def _activation(act):
    kind = ACTIVATIONS.get(act)
    if kind is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, not {act!r}")
    return kind


def tn_gated(A, Bt, offsets=None, act="silu", keep=False, H=None, P=None, stream=None):
    """Gated projections: P^T[t] = A Bt[t] for A's M gate and M up rows, H^T[t, m] =
    act(P^T[t, m]) P^T[t, M + m].  A (2 M, K) and Bt (T, K), or A (E, 2 M, K) and
    offsets (E + 1,) int32 as in tn_grouped; all fp16 or all bf16, rows contiguous ->
    H (T, M).  keep: returns (H, P) with the fp32 products P (T, 2 M), which
    tn_gated_grad takes.  act: "silu", "gelu" or "gelu_tanh"."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt)
    dtype, device = A.dtype, A.device
    half, kind = _half_type(dtype, "A"), _activation(act)
    E, M, K, T, lda, stride_a, ldb, _, _ = _gated_operands(A, Bt, offsets)
    if _elsewhere(device.index):
        with torch.cuda.device(device):
            return tn_gated(A, Bt, offsets, act, keep, H, P, stream)
    H, ldh = _result(H, (T, M), dtype, device, stream, "H")
    ldp = 0
    if keep or P is not None:
        P, ldp = _result(P, (T, 2 * M), torch.float32, device, stream, "P")
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_gated_workspace(0, offsets is None, E, M, K, T, a, lda, stride_a, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    _check(calls.gemm_tn_gated(half, kind, E, M, K, T, a, lda, stride_a, b, ldb, _ptr(offsets), H.data_ptr(), ldh, _ptr(P),
                               ldp, held.data_ptr() if n > 0 else None, n, _launch_stream(device.index, stream)))
    return H if P is None else (H, P)


def tn_gated_grad(A, Bt, P, dHt, offsets=None, act="silu", dA=None, dBt=None, want_a=True, want_b=True, stream=None):
    """The gradients of tn_gated: from its operands, its products P and the gradient
    dHt (T, M) of its result -> (dA of A's shape, dBt (T, K)).  want_a, want_b: a
    gradient that is not wanted is not computed, and None.  Rows of dBt that belong to
    no expert are not written; an expert without rows has zeros in dA."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, P, dHt)
    dtype, device = A.dtype, A.device
    half, kind = _half_type(dtype, "A"), _activation(act)
    E, M, K, T, lda, stride_a, ldb, ldp, lddh = _gated_operands(A, Bt, offsets, P, dHt)
    if _elsewhere(device.index):
        with torch.cuda.device(device):
            return tn_gated_grad(A, Bt, P, dHt, offsets, act, dA, dBt, want_a, want_b, stream)
    ldda = stride_da = lddb = 0
    if want_a:
        if dA is None:
            dA = _empty(A.shape, dtype, device, stream)
            ldda, stride_da = max(K, 1), 2 * M * K if E > 1 else 0
        elif offsets is None:
            ldda = _rows(dA, dtype, "dA", tuple(A.shape))
        else:
            ldda, stride_da = _experts(dA, dtype, "dA", tuple(A.shape))
        _same_device(device, dA=dA)
    if want_b:
        dBt, lddb = _result(dBt, (T, K), dtype, device, stream, "dBt")
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_gated_workspace(1, offsets is None, E, M, K, T, a, lda, stride_a, b, ldb)
    held = _workspace(device, stream, n if offsets is None else n + _BEHIND_MAPS) if n > 0 else None
    _check(calls.gemm_tn_gated_grad(half, kind, E, M, K, T, a, lda, stride_a, b, ldb, _ptr(offsets), P.data_ptr(), ldp,
                                    dHt.data_ptr(), lddh, dA.data_ptr() if want_a else None, ldda, stride_da,
                                    dBt.data_ptr() if want_b else None, lddb, held.data_ptr() if n > 0 else None, n,
                                    _launch_stream(device.index, stream)))
    return (dA if want_a else None), (dBt if want_b else None)


def _result(t, shape, dtype, device, stream, name):
    """(t, its row stride): a new tensor on the call's stream, or the caller's."""
    if t is None:
        return _empty(shape, dtype, device, stream), max(shape[1], 1)
    ld = _rows(t, dtype, name, shape)
    _same_device(device, **{name: t})
    return t, ld


def _loss_operands(A, Bt, **vectors):
    """(GEMM_IN_..., M, N, K, lda, ldb) of a vocabulary A (M, K), tokens Bt (N, K) and what belongs to the tokens."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, *vectors.values())
    half, sa, sb = _half_type(A.dtype, "A"), A.shape, Bt.shape
    if len(sa) == 2 == len(sb) and sa[1] == sb[1] > 0 < sa[0] and Bt.dtype is A.dtype and _plain(torch, A, Bt, *vectors.values()):
        for name, t in vectors.items():
            if t.dim() != 1 or t.shape[0] != sb[0] or t.dtype is not (torch.int64 if name == "targets" else torch.float32):
                break
        else:
            return half, sa[0], sb[0], sa[1], sa[1], sa[1]
    lda, ldb = _rows(A, A.dtype, "A", cuda=False), _rows(Bt, A.dtype, "Bt", cuda=False)
    (M, K), N = A.shape, Bt.shape[0]
    if Bt.shape[1] != K:
        raise ValueError(f"A is {tuple(A.shape)} and Bt {tuple(Bt.shape)}: their second dimensions (K) differ")
    if M == 0 and N > 0:
        raise ValueError("A has no rows: there are no classes")
    for name, t in vectors.items():
        _vector(t, torch.int64 if name == "targets" else torch.float32, N, name)
    _same_device(A.device, Bt=Bt, **vectors)
    return half, M, N, K, lda, ldb


def tn_cross_entropy(A, Bt, targets, stream=None):
    """Softmax cross entropy of Bt's rows against the classes A: A (M, K) and Bt (N, K),
    both fp16 or both bf16, targets (N,) int64 -> (loss (N,), lse (N,)), fp32: lse[n] =
    log sum_m exp(A[m] . Bt[n]), loss[n] = lse[n] - A[targets[n]] . Bt[n]; 0 for a
    negative target, NaN for one of M or more.  The logits are never held."""
    half, M, N, K, lda, ldb = _loss_operands(A, Bt, targets=targets)
    torch, device = _torch, A.device
    if _elsewhere(device.index):
        with torch.cuda.device(device):
            return tn_cross_entropy(A, Bt, targets, stream)
    loss, lse = (_empty((N,), torch.float32, device, stream) for _ in range(2))
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_cross_entropy_workspace(0, M, N, K, a, lda, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    _check(calls.gemm_tn_cross_entropy(half, M, N, K, a, lda, b, ldb, targets.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                                       held.data_ptr() if n > 0 else None, n, _launch_stream(device.index, stream)))
    return loss, lse


def tn_cross_entropy_grad(A, Bt, targets, lse, dloss, dA=None, dBt=None, want_a=True, want_b=True, stream=None):
    """The gradients of tn_cross_entropy's loss: from its operands, its lse and the
    gradient dloss (N,) fp32 of the loss -> (dA (M, K), dBt (N, K)).  want_a, want_b: a
    gradient that is not wanted is not computed, and None."""
    half, M, N, K, lda, ldb = _loss_operands(A, Bt, targets=targets, lse=lse, dloss=dloss)
    torch, device = _torch, A.device
    if _elsewhere(device.index):
        with torch.cuda.device(device):
            return tn_cross_entropy_grad(A, Bt, targets, lse, dloss, dA, dBt, want_a, want_b, stream)
    ldda = lddb = 0
    if want_a:
        dA, ldda = _result(dA, (M, K), A.dtype, device, stream, "dA")
    if want_b:
        dBt, lddb = _result(dBt, (N, K), A.dtype, device, stream, "dBt")
    a, b = A.data_ptr(), Bt.data_ptr()
    n = calls.gemm_cross_entropy_workspace(1, M, N, K, a, lda, b, ldb)
    held = _workspace(device, stream, n) if n > 0 else None
    _check(calls.gemm_tn_cross_entropy_grad(half, M, N, K, a, lda, b, ldb, targets.data_ptr(), lse.data_ptr(),
                                            dloss.data_ptr(), dA.data_ptr() if want_a else None, ldda,
                                            dBt.data_ptr() if want_b else None, lddb, held.data_ptr() if n > 0 else None, n,
                                            _launch_stream(device.index, stream)))
    return (dA if want_a else None), (dBt if want_b else None)


# ---------------------------------------------------------------- 4-bit weights
def w4_tn(A, Bt, scale_a, group, C=None, stream=None):
    """C^T[n, m] = sum over groups g of scale_a[m, g] (sum over k in g of q[m, k] Bt[n, k]):
    A (M, ceil(K / 2)) uint8, two signed 4-bit integers a byte, the even k in the low
    half; Bt (N, K) and scale_a (M, ceil(K / group)) both fp16 or both bf16; group 32, 64,
    128 or 256 terms -> (N, M) of their type.  For the few tokens of a decode step."""
    torch = _torch or _load_torch()
    _tensors(torch, A, Bt, scale_a)
    dtype, device, sa, sb, ss = Bt.dtype, A.device, A.shape, Bt.shape, scale_a.shape
    half = _half_type(dtype, "Bt")
    if group not in (32, 64, 128, 256):
        raise ValueError(f"group must be 32, 64, 128 or 256, not {group!r}")
    if (C is None and A.dtype is torch.uint8 and scale_a.dtype is dtype and len(sa) == 2 == len(sb) and len(ss) == 2
            and 0 < sa[1] == (sb[1] + 1) // 2 and sa[0] == ss[0] and ss[1] == -(-sb[1] // group)
            and A.stride(1) == 1 and sa[0] > 1 and A.get_device() == Bt.get_device() and _plain(torch, Bt, scale_a)):
        M, (N, K) = sa[0], sb
        lda, ldb, lds = A.stride(0), K, ss[1]
        C, ldc = _empty((N, M), dtype, device, stream), M
    else:
        lda = _rows(A, torch.uint8, "A", cuda=False)
        ldb = _rows(Bt, dtype, "Bt", cuda=False)
        M, (N, K) = A.shape[0], Bt.shape
        if A.shape[1] != (K + 1) // 2:
            raise ValueError(f"A has {A.shape[1]} bytes a row, {(K + 1) // 2} hold {K} terms")
        lds = _rows(scale_a, dtype, "scale_a", (M, -(-K // group)), cuda=False)
        _same_device(device, Bt=Bt, scale_a=scale_a)
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return w4_tn(A, Bt, scale_a, group, C, stream)
        C, ldc = _result(C, (N, M), dtype, device, stream, "C")
    _check(calls.gemm_w4_tn(half, M, N, K, A.data_ptr(), lda, scale_a.data_ptr(), lds, group, Bt.data_ptr(), ldb,
                            C.data_ptr(), ldc, _launch_stream(device.index, stream)))
    return C


def quantize_w4_rows(x, group, dtype=None, stream=None):
    """x: a 2-D float32 / float16 / bfloat16 CUDA tensor with unit column stride.  Returns
    (codes (rows, ceil(cols / 2)) uint8, scale (rows, ceil(cols / group)) of `dtype`):
    w4_tn's A and scale_a.  dtype: torch.float16 or torch.bfloat16 (x's own, unless it
    is float32).  The codes' rows start on 16-byte boundaries."""
    torch = _torch or _load_torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D float32/float16/bfloat16 tensor")
    xtype, device = x.dtype, x.device
    kind = GEMM_IN_F32 if xtype is torch.float32 else _half_kinds.get(xtype)
    if kind is None:
        raise ValueError("x must be a 2-D float32/float16/bfloat16 tensor")
    if dtype is None:
        if xtype is torch.float32:
            raise ValueError("dtype must say which 16-bit type the scales of a float32 tensor have")
        dtype = xtype
    half = _half_type(dtype, "dtype")
    if group not in (32, 64, 128, 256):
        raise ValueError(f"group must be 32, 64, 128 or 256, not {group!r}")
    rows, cols = x.shape
    if cols > 0 and _plain(torch, x):
        ldx = cols
    else:
        ldx = _rows(x, xtype, "x")
        if _elsewhere(device.index):
            with torch.cuda.device(device):
                return quantize_w4_rows(x, group, dtype, stream)
    row_bytes, groups = (cols + 1) // 2, -(-cols // group)
    ldq = max(-(-row_bytes // 16) * 16, 1)
    q = _empty((rows, ldq), torch.uint8, device, stream)
    if ldq != row_bytes:
        q = q[:, :row_bytes]
    scale = _empty((rows, groups), dtype, device, stream)
    _check(calls.gemm_quantize_w4_rows(x.data_ptr(), kind, rows, cols, ldx, group, q.data_ptr(), ldq, half, scale.data_ptr(),
                                       max(groups, 1), _launch_stream(device.index, stream)))
    return q, scale
