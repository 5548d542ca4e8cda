"""ctypes binding of ``libgemm_f32.so`` (the C ABI in ``include/gemm_f32.h``).

Two layers, both argument marshalling only -- every step of the product runs
in the HIP kernels:

* functions named exactly as the C entry points (``gemm_f32``,
  ``gemm_f32_ref_gpu``, ...) taking plain integers: sizes, device pointers,
  pitches and a ``hipStream_t`` as an integer (0 = default stream);
* ``gemm`` / ``gemm_ref`` / ``run_kernel``: the same calls on torch tensors,
  which read sizes, pitches and pointers from the tensors and enqueue on
  torch's current stream of the tensors' device.

There is no fallback: if the library is missing, ``load()`` raises.  The
environment variable ``GEMM_F32_LIB`` names another build of the same library
to load instead (the host-sanitizer build of ``sanitize_host.py``).
"""
from __future__ import annotations

import ctypes
import os
from array import array
from pathlib import Path

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libgemm_f32.so"

GEMM_F32_OK = 0
STATUS_NAMES = {
    0: "GEMM_F32_OK", 1: "GEMM_F32_ERR_INVALID_DIM", 2: "GEMM_F32_ERR_INVALID_LD",
    3: "GEMM_F32_ERR_NULL_PTR", 4: "GEMM_F32_ERR_ALIAS", 5: "GEMM_F32_ERR_DEVICE",
    6: "GEMM_F32_ERR_WORKSPACE", 7: "GEMM_F32_ERR_LAUNCH", 8: "GEMM_F32_ERR_BAD_KERNEL",
    9: "GEMM_F32_ERR_POINTER", 10: "GEMM_F32_ERR_INVALID_ARG", 11: "GEMM_F32_ERR_SCRATCH",
}
ACT_NONE, ACT_RELU = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
Q4_INT, Q4_E2M1 = 0, 1
SCALE_F32, SCALE_F16, SCALE_BF16, SCALE_E8M0 = 0, 1, 2, 3
EXPORTS = ["gemm_f32", "gemm_f32_ex", "gemm_f32_ref_gpu", "gemm_f32_status_string",
           "gemm_f32_selected_kernel", "gemm_f32_selected_kernel_ex", "gemm_f32_version",
           "gemm_f32_kernel_count", "gemm_f32_kernel_name", "gemm_f32_run_kernel",
           "gemm_f32_run_kernel_ex", "gemm_f32_release_workspaces", "gemm_f32_batched",
           "gemm_f32_selected_kernel_batched", "reduce_sum_f32", "gemm_f32_fused",
           "gemm_f32_run_kernel_fused", "gemm_f32_noalloc", "gemm_f32_clock_probe",
           "gemm_f32_group_rows", "gemm_f32_grouped", "gemm_f32_grouped_wgrad",
           "gemm_f32_adapters", "gemm_f32_route", "gemm_f32_route_grad", "gemm_f32_join_rows",
           "gemm_f32_join_rows_grad", "gemm_f32_q4", "gemm_f32_q4_grouped", "gemm_f32_norm",
           "gemm_f32_clip"]
MAX_GROUPS = 1024
MAX_TOP = 64
CLOCK_PROBE_WORKGROUPS = 1024


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({gemm_f32_status_string(status)})")


_lib = None


def load(lib_path=None):
    """Load the HIP library (once; ``lib_path`` picks another build of it,
    such as the sweep library of tune.py).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        if lib_path is not None and Path(lib_path) != Path(_lib._name):
            raise RuntimeError(f"{_lib._name} is already loaded")
        return _lib
    if lib_path is None and os.environ.get("GEMM_F32_LIB"):
        lib_path = os.environ["GEMM_F32_LIB"]
    path = Path(lib_path) if lib_path is not None else LIB_PATH
    if not path.exists():
        raise FileNotFoundError(
            f"{path} is missing: build it with `python -m dense_fp32_gemm_f32_amd.build_lib` "
            "(there is no CPU or PyTorch fallback)")
    lib = ctypes.CDLL(str(path))
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    gemm_args = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    for name in ("gemm_f32", "gemm_f32_ref_gpu", "gemm_f32_noalloc"):
        getattr(lib, name).argtypes = gemm_args
        getattr(lib, name).restype = ctypes.c_int
    lib.gemm_f32_run_kernel.argtypes = [ctypes.c_int, *gemm_args]
    lib.gemm_f32_run_kernel.restype = ctypes.c_int
    f32, ci = ctypes.c_float, ctypes.c_int
    ex_args = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.gemm_f32_ex.argtypes = ex_args
    lib.gemm_f32_ex.restype = ctypes.c_int
    lib.gemm_f32_run_kernel_ex.argtypes = [ci, *ex_args]
    lib.gemm_f32_run_kernel_ex.restype = ctypes.c_int
    fused_args = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp, ci, vp]
    lib.gemm_f32_fused.argtypes = fused_args
    lib.gemm_f32_fused.restype = ctypes.c_int
    lib.gemm_f32_run_kernel_fused.argtypes = [ci, *fused_args]
    lib.gemm_f32_run_kernel_fused.restype = ctypes.c_int
    lib.gemm_f32_selected_kernel_ex.argtypes = [ci, ci, i64, i64, i64, i64, i64, i64, f32, f32,
                                                vp, vp, vp]
    lib.gemm_f32_selected_kernel_ex.restype = ctypes.c_char_p
    lib.gemm_f32_status_string.argtypes = [ctypes.c_int]
    lib.gemm_f32_status_string.restype = ctypes.c_char_p
    lib.gemm_f32_selected_kernel.argtypes = [i64, i64, i64, i64, i64, i64, vp, vp, vp]
    lib.gemm_f32_selected_kernel.restype = ctypes.c_char_p
    lib.gemm_f32_version.argtypes = []
    lib.gemm_f32_version.restype = ctypes.c_int
    lib.gemm_f32_kernel_count.argtypes = []
    lib.gemm_f32_kernel_count.restype = ctypes.c_int
    lib.gemm_f32_kernel_name.argtypes = [ctypes.c_int]
    lib.gemm_f32_kernel_name.restype = ctypes.c_char_p
    lib.gemm_f32_release_workspaces.argtypes = []
    lib.gemm_f32_release_workspaces.restype = ctypes.c_int
    lib.gemm_f32_clock_probe.argtypes = [i64, vp, vp, vp, vp]
    lib.gemm_f32_clock_probe.restype = ctypes.c_int
    lib.reduce_sum_f32.argtypes = [i64, vp, vp, vp]
    lib.reduce_sum_f32.restype = ctypes.c_int
    lib.gemm_f32_batched.argtypes = [i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64,
                                     i64, vp]
    lib.gemm_f32_batched.restype = ctypes.c_int
    lib.gemm_f32_selected_kernel_batched.argtypes = [i64, i64, i64, i64, i64, i64, i64, i64,
                                                     i64, vp, vp]
    lib.gemm_f32_selected_kernel_batched.restype = ctypes.c_char_p
    lib.gemm_f32_group_rows.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp]
    lib.gemm_f32_group_rows.restype = ci
    lib.gemm_f32_grouped.argtypes = [ci, i64, i64, i64, i64, vp, f32, vp, i64, i64, vp,
                                     vp, i64, i64, f32, vp, i64, i64, vp, vp, i64, ci, vp]
    lib.gemm_f32_grouped.restype = ci
    lib.gemm_f32_grouped_wgrad.argtypes = [i64, i64, i64, i64, vp, f32, vp, i64, i64, vp,
                                           vp, i64, i64, vp, f32, vp, i64, i64, vp]
    lib.gemm_f32_grouped_wgrad.restype = ci
    lib.gemm_f32_adapters.argtypes = [ci, i64, i64, i64, i64, i64, i64, vp, vp, vp, vp, i64,
                                      vp, i64, vp, i64, i64, vp, i64, i64, vp, vp, i64, vp, i64,
                                      vp]
    lib.gemm_f32_adapters.restype = ci
    lib.gemm_f32_route.argtypes = [i64, i64, i64, vp, i64, vp, ci, i64, i64, ci, ci, f32, vp, vp,
                                   vp]
    lib.gemm_f32_route.restype = ci
    lib.gemm_f32_route_grad.argtypes = [i64, i64, i64, vp, i64, ci, ci, f32, vp, vp, vp, i64, vp]
    lib.gemm_f32_route_grad.restype = ci
    lib.gemm_f32_join_rows.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, f32, vp, i64, vp]
    lib.gemm_f32_join_rows.restype = ci
    lib.gemm_f32_join_rows_grad.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64,
                                            vp, vp]
    lib.gemm_f32_join_rows_grad.restype = ci
    lib.gemm_f32_q4.argtypes = [i64, i64, i64, f32, vp, i64, ci, i64, vp, i64, ci, vp, i64, vp,
                                i64, f32, vp, i64, vp, ci, vp]
    lib.gemm_f32_q4.restype = ci
    lib.gemm_f32_q4_grouped.argtypes = [i64, i64, i64, i64, vp, f32, vp, i64, i64, vp, ci, i64, vp,
                                        i64, i64, ci, vp, i64, i64, vp, i64, i64, f32, vp, i64,
                                        i64, vp, vp, i64, ci, vp]
    lib.gemm_f32_q4_grouped.restype = ci
    lib.gemm_f32_norm.argtypes = [i64, vp, vp, vp, vp]
    lib.gemm_f32_norm.restype = ci
    lib.gemm_f32_clip.argtypes = [i64, vp, vp, vp, f32, vp, vp]
    lib.gemm_f32_clip.restype = ci
    _lib = lib
    return lib


# ---- the C entry points, same names, plain integers ------------------------

def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                              stream)


def gemm_f32_fused(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                   stream=0) -> int:
    return load().gemm_f32_fused(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                 bias, act, stream)


def gemm_f32_run_kernel_fused(index, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                              ldc, bias, act, stream=0) -> int:
    return load().gemm_f32_run_kernel_fused(index, transA, transB, M, N, K, alpha, A, lda, B,
                                            ldb, beta, C, ldc, bias, act, stream)


def gemm_f32_run_kernel_ex(index, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                           stream=0) -> int:
    return load().gemm_f32_run_kernel_ex(index, transA, transB, M, N, K, alpha, A, lda, B, ldb,
                                         beta, C, ldc, stream)


def gemm_f32_selected_kernel_ex(transA, transB, M, N, K, lda, ldb, ldc, alpha=1.0, beta=0.0,
                                A=0, B=0, C=0) -> str:
    return load().gemm_f32_selected_kernel_ex(transA, transB, M, N, K, lda, ldb, ldc, alpha,
                                              beta, A, B, C).decode()


def gemm_f32_batched(M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch,
                     stream=0) -> int:
    return load().gemm_f32_batched(M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC,
                                   batch, stream)


def gemm_f32_selected_kernel_batched(M, N, K, lda, strideA, ldb, strideB, ldc, batch, A=0,
                                     B=0) -> str:
    return load().gemm_f32_selected_kernel_batched(M, N, K, lda, strideA, ldb, strideB, ldc,
                                                   batch, A, B).decode()


def gemm_f32_clock_probe(iters, stamps, wall_khz=None, max_khz=None, stream=0) -> int:
    return load().gemm_f32_clock_probe(iters, stamps, wall_khz, max_khz, stream)


def reduce_sum_f32(n, x, out, stream=0) -> int:
    return load().reduce_sum_f32(n, x, out, stream)


def gemm_f32_group_rows(n, groups, per_row, index, offsets, order, rows, stream=0) -> int:
    return load().gemm_f32_group_rows(n, groups, per_row, index, offsets, order, rows, stream)


def gemm_f32_grouped(transB, rows, N, K, groups, offsets, alpha, A, lda, rowsA, indexA, B, ldb,
                     strideB, beta, C, ldc, rowsC, indexC, bias, strideBias, act,
                     stream=0) -> int:
    return load().gemm_f32_grouped(transB, rows, N, K, groups, offsets, alpha, A, lda, rowsA,
                                   indexA, B, ldb, strideB, beta, C, ldc, rowsC, indexC, bias,
                                   strideBias, act, stream)


def gemm_f32_grouped_wgrad(rows, M, N, groups, offsets, alpha, A, lda, rowsA, indexA, B, ldb,
                           rowsB, indexB, beta, C, ldc, strideC, stream=0) -> int:
    return load().gemm_f32_grouped_wgrad(rows, M, N, groups, offsets, alpha, A, lda, rowsA,
                                         indexA, B, ldb, rowsB, indexB, beta, C, ldc, strideC,
                                         stream)


def gemm_f32_adapters(trans, M, N, K, R, groups, places, offsets, order, scale, X, ldx, W, ldw,
                      D, ldd, strideD, U, ldu, strideU, bias, H, ldh, Y, ldy, stream=0) -> int:
    return load().gemm_f32_adapters(trans, M, N, K, R, groups, places, offsets, order, scale, X,
                                    ldx, W, ldw, D, ldd, strideD, U, ldu, strideU, bias, H, ldh,
                                    Y, ldy, stream)


def gemm_f32_route(tokens, experts, top, logits, ldl, bias, score, groups, group_top, group_best,
                   renorm, scale, choice, weight, stream=0) -> int:
    return load().gemm_f32_route(tokens, experts, top, logits, ldl, bias, score, groups, group_top,
                                 group_best, renorm, scale, choice, weight, stream)


def gemm_f32_route_grad(tokens, experts, top, logits, ldl, score, renorm, scale, choice, dweight,
                        dlogits, lddl, stream=0) -> int:
    return load().gemm_f32_route_grad(tokens, experts, top, logits, ldl, score, renorm, scale,
                                      choice, dweight, dlogits, lddl, stream)


def gemm_f32_join_rows(tokens, top, N, H, ldh, weight, choice, groups, beta, Y, ldy,
                       stream=0) -> int:
    return load().gemm_f32_join_rows(tokens, top, N, H, ldh, weight, choice, groups, beta, Y, ldy,
                                     stream)


def gemm_f32_join_rows_grad(tokens, top, N, dY, lddy, H, ldh, weight, choice, groups, dH, lddh,
                            dweight, stream=0) -> int:
    return load().gemm_f32_join_rows_grad(tokens, top, N, dY, lddy, H, ldh, weight, choice, groups,
                                          dH, lddh, dweight, stream)


def gemm_f32_q4(M, N, K, alpha, A, lda, format, group, codes, ldq, scale_type, scale, lds, zero,
                ldz, beta, C, ldc, bias, act, stream=0) -> int:
    return load().gemm_f32_q4(M, N, K, alpha, A, lda, format, group, codes, ldq, scale_type, scale,
                              lds, zero, ldz, beta, C, ldc, bias, act, stream)


def gemm_f32_q4_grouped(rows, N, K, groups, offsets, alpha, A, lda, rowsA, indexA, format, group,
                        codes, ldq, strideQ, scale_type, scale, lds, strideS, zero, ldz, strideZ,
                        beta, C, ldc, rowsC, indexC, bias, strideBias, act, stream=0) -> int:
    return load().gemm_f32_q4_grouped(rows, N, K, groups, offsets, alpha, A, lda, rowsA, indexA,
                                      format, group, codes, ldq, strideQ, scale_type, scale, lds,
                                      strideS, zero, ldz, strideZ, beta, C, ldc, rowsC, indexC,
                                      bias, strideBias, act, stream)


def gemm_f32_norm(count, x, n, norm, stream=0) -> int:
    return load().gemm_f32_norm(count, x, n, norm, stream)


def gemm_f32_clip(count, x, n, out, max_norm, norm, stream=0) -> int:
    return load().gemm_f32_clip(count, x, n, out, max_norm, norm, stream)


def gemm_f32_ref_gpu(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f32_ref_gpu(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_run_kernel(index, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f32_run_kernel(index, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_status_string(status: int) -> str:
    return load().gemm_f32_status_string(int(status)).decode()


def gemm_f32_selected_kernel(M, N, K, lda, ldb, ldc, A=0, B=0, C=0) -> str:
    return load().gemm_f32_selected_kernel(M, N, K, lda, ldb, ldc, A, B, C).decode()


def gemm_f32_version() -> int:
    return load().gemm_f32_version()


def gemm_f32_kernel_count() -> int:
    return load().gemm_f32_kernel_count()


def gemm_f32_kernel_name(index: int) -> str | None:
    r = load().gemm_f32_kernel_name(index)
    return None if r is None else r.decode()


def gemm_f32_release_workspaces() -> int:
    return load().gemm_f32_release_workspaces()


def kernel_names() -> list[str]:
    return [gemm_f32_kernel_name(i) for i in range(gemm_f32_kernel_count())]


def kernel_index(name: str) -> int:
    names = kernel_names()
    if name not in names:
        raise KeyError(f"no kernel named {name!r}")
    return names.index(name)


# ---- torch tensors -----------------------------------------------------------

def _pitch(t, name):
    import torch
    if t.dtype != torch.float32 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32 tensor")
    if t.device.type != "cuda":
        raise TypeError(f"{name} must be on a GPU (got {t.device})")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")
    if t.shape[0] > 1 and t.shape[1] > 0 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} rows must not overlap (stride(0) >= the row length); an "
                         "expanded tensor needs .contiguous()")
    return max(t.stride(0), t.shape[1], 1) if t.shape[0] > 1 else max(t.shape[1], 1)


def _args(A, B, C):
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner sizes differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {M}x{N}, got {tuple(C.shape)}")
    lda, ldb, ldc = _pitch(A, "A"), _pitch(B, "B"), _pitch(C, "C")
    if not (A.device == B.device == C.device):
        raise ValueError("A, B and C must be on one device")
    stream = torch.cuda.current_stream(A.device).cuda_stream
    return (M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(), ldc, stream), C


def gemm(A, B, C=None):
    """C = A @ B on the GPU with the dispatcher's kernel; returns C."""
    args, C = _args(A, B, C)
    with _device(A):
        rc = gemm_f32(*args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32")
    return C


def gemm_noalloc(A, B, C=None):
    """C = A @ B through gemm_f32_noalloc (the fixed scratch array, no
    allocation inside the library); returns C."""
    args, C = _args(A, B, C)
    with _device(A):
        rc = gemm_f32_noalloc(*args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_noalloc")
    return C


def gemm_ref(A, B, C=None):
    """C = A @ B with the naive reference kernel; returns C."""
    args, C = _args(A, B, C)
    with _device(A):
        rc = gemm_f32_ref_gpu(*args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_ref_gpu")
    return C


def run_kernel(index_or_name, A, B, C=None):
    """C = A @ B with one named (or indexed) kernel of the table; returns C."""
    index = kernel_index(index_or_name) if isinstance(index_or_name, str) else int(index_or_name)
    args, C = _args(A, B, C)
    with _device(A):
        rc = gemm_f32_run_kernel(index, *args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, f"gemm_f32_run_kernel({index_or_name})")
    return C


def _args_batched(A, B, C):
    """Sizes, pointers, pitches and batch strides of 3-D tensors (batch, rows,
    cols); a batch stride of 0 (an expanded tensor) shares one matrix."""
    import torch
    if A.dim() != 3 or B.dim() != 3:
        raise TypeError("A and B must be 3-D (batch, rows, cols)")
    batch, M, K = A.shape
    batch2, K2, N = B.shape
    if K != K2 or batch != batch2:
        raise ValueError(f"shapes differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    if C is None:
        C = torch.empty((batch, M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (batch, M, N):
        raise ValueError(f"C must be {batch}x{M}x{N}, got {tuple(C.shape)}")
    if batch == 0:
        lda, ldb, ldc = max(K, 1), max(N, 1), max(N, 1)
    else:
        lda, ldb, ldc = _pitch(A[0], "A"), _pitch(B[0], "B"), _pitch(C[0], "C")
    sa, sb, sc = A.stride(0), B.stride(0), C.stride(0)
    if not (A.device == B.device == C.device):
        raise ValueError("A, B and C must be on one device")
    stream = torch.cuda.current_stream(A.device).cuda_stream
    return (M, N, K, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, C.data_ptr(), ldc, sc,
            batch, stream), C


def gemm_batched(A, B, C=None):
    """C[b] = A[b] @ B[b] for every b, in as few launches as possible (3-D
    tensors; a stride of 0 along the batch shares one matrix).  Returns C."""
    args, C = _args_batched(A, B, C)
    with _device(A):
        rc = gemm_f32_batched(*args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_batched")
    return C


def selected_kernel_batched(A, B, C=None) -> str:
    (M, N, K, a, lda, sa, b, ldb, sb, _c, ldc, _sc, batch, _s), _ = _args_batched(A, B, C)
    return gemm_f32_selected_kernel_batched(M, N, K, lda, sa, ldb, sb, ldc, batch, a, b)


def reduce_sum(x, out=None):
    """Sum of a 1-D contiguous float32 GPU tensor into a 1-element tensor
    (returned), in an order fixed by the length."""
    import torch
    if x.dtype != torch.float32 or x.dim() != 1 or (x.numel() > 1 and x.stride(0) != 1):
        raise TypeError("x must be a contiguous 1-D float32 tensor")
    if x.device.type != "cuda":
        raise TypeError(f"x must be on a GPU (got {x.device})")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    with _device(x):
        rc = reduce_sum_f32(x.numel(), x.data_ptr(), out.data_ptr(), stream)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "reduce_sum_f32")
    return out


def clock_probe(iters=2400, device=None):
    """Run gemm_f32_clock_probe on torch's current stream of ``device`` and
    wait for it.  Returns (per-workgroup achieved shader clocks in GHz, the
    constant counter's rate in kHz, the device's peak shader clock in kHz)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    stamps = torch.zeros(4 * CLOCK_PROBE_WORKGROUPS, dtype=torch.int64, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    wall, peak = ctypes.c_int(0), ctypes.c_int(0)
    with _device(stamps):
        rc = gemm_f32_clock_probe(iters, stamps.data_ptr(), ctypes.byref(wall),
                                  ctypes.byref(peak), stream)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_clock_probe")
    torch.cuda.synchronize(dev)
    w = stamps.view(-1, 4).cpu().tolist()
    ghz = [wall.value * 1e-6 * (t1 - t0) / (r1 - r0) for t0, r0, t1, r1 in w if r1 > r0]
    return ghz, wall.value, peak.value


def _args_ex(A, B, C, trans_a, trans_b):
    import torch
    M, K = (A.shape[1], A.shape[0]) if trans_a else tuple(A.shape)
    K2, N = (B.shape[1], B.shape[0]) if trans_b else tuple(B.shape)
    if K != K2:
        raise ValueError(f"inner sizes differ: op(A) is {M}x{K}, op(B) is {K2}x{N}")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {M}x{N}, got {tuple(C.shape)}")
    lda, ldb, ldc = _pitch(A, "A"), _pitch(B, "B"), _pitch(C, "C")
    if not (A.device == B.device == C.device):
        raise ValueError("A, B and C must be on one device")
    stream = torch.cuda.current_stream(A.device).cuda_stream
    return (M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(), ldc, stream), C


def gemm_ex(A, B, C=None, *, trans_a=False, trans_b=False, alpha=1.0, beta=0.0, kernel=None):
    """C = alpha * op(A) @ op(B) + beta * C on the GPU; A and B are the stored
    matrices (A is K x M when trans_a, B is N x K when trans_b).  ``kernel``
    runs one named (or indexed) kernel of the table instead of the
    dispatcher's.  Returns C."""
    (M, N, K, a, lda, b, ldb, c, ldc, stream), C = _args_ex(A, B, C, trans_a, trans_b)
    ta, tb = int(bool(trans_a)), int(bool(trans_b))
    with _device(A):
        if kernel is None:
            rc = gemm_f32_ex(ta, tb, M, N, K, alpha, a, lda, b, ldb, beta, c, ldc, stream)
        else:
            index = kernel_index(kernel) if isinstance(kernel, str) else int(kernel)
            rc = gemm_f32_run_kernel_ex(index, ta, tb, M, N, K, alpha, a, lda, b, ldb, beta, c,
                                        ldc, stream)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_ex" if kernel is None else f"gemm_f32_run_kernel_ex({kernel})")
    return C


def gemm_fused(A, B, C=None, *, trans_a=False, trans_b=False, alpha=1.0, beta=0.0, bias=None,
               act=ACT_NONE, kernel=None):
    """C = act(alpha * op(A) @ op(B) + beta * C + bias) on the GPU; ``bias`` a
    1-D contiguous tensor of N floats (or None), ``act`` ACT_NONE or ACT_RELU.
    ``kernel`` runs one named (or indexed) kernel of the table.  Returns C."""
    (M, N, K, a, lda, b, ldb, c, ldc, stream), C = _args_ex(A, B, C, trans_a, trans_b)
    bptr = 0
    if bias is not None:
        if bias.dim() != 1 or bias.numel() != N or (N > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be a contiguous vector of {N} floats")
        bptr = bias.data_ptr()
    ta, tb = int(bool(trans_a)), int(bool(trans_b))
    with _device(A):
        if kernel is None:
            rc = gemm_f32_fused(ta, tb, M, N, K, alpha, a, lda, b, ldb, beta, c, ldc, bptr,
                                int(act), stream)
        else:
            index = kernel_index(kernel) if isinstance(kernel, str) else int(kernel)
            rc = gemm_f32_run_kernel_fused(index, ta, tb, M, N, K, alpha, a, lda, b, ldb, beta,
                                           c, ldc, bptr, int(act), stream)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_fused" if kernel is None else
                        f"gemm_f32_run_kernel_fused({kernel})")
    return C


def selected_kernel_ex(A, B, C=None, *, trans_a=False, trans_b=False, alpha=1.0,
                       beta=0.0) -> str:
    M, K = (A.shape[1], A.shape[0]) if trans_a else tuple(A.shape)
    N = B.shape[0] if trans_b else B.shape[1]
    lda = max(A.stride(0), A.shape[1], 1)
    ldb = max(B.stride(0), B.shape[1], 1)
    ldc = N if C is None else max(C.stride(0), N)
    return gemm_f32_selected_kernel_ex(int(bool(trans_a)), int(bool(trans_b)), M, N, K, lda,
                                       ldb, max(ldc, 1), alpha, beta, A.data_ptr(),
                                       B.data_ptr(), 0 if C is None else C.data_ptr())


def selected_kernel(A, B, C=None) -> str:
    M, K = A.shape
    N = B.shape[1]
    ldc = N if C is None else max(C.stride(0), N)
    return gemm_f32_selected_kernel(M, N, K, max(A.stride(0), K, 1), max(B.stride(0), N, 1),
                                    max(ldc, 1), A.data_ptr(), B.data_ptr(),
                                    0 if C is None else C.data_ptr())


# ---- grouped products --------------------------------------------------------
# (short calls: the checks below read each tensor's sizes and strides once)

def _on(t, call, *args):
    """call(*args, stream) with t's device current, on torch's current stream of it."""
    import torch
    index = t.device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        return call(*args, stream)
    with _device(t):
        return call(*args, stream)


def _index(t, name, device, count=None):
    """Pointer of a contiguous 1-D int32 tensor on ``device`` (0 for None)."""
    import torch
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D int32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if count is not None and t.shape[0] != count:
        raise ValueError(f"{name} must have {count} entries, got {t.shape[0]}")
    return t.data_ptr()


def _rows(rows, cols, s0, s1, name):
    """Pitch of a rows x cols matrix with these strides."""
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} rows must be contiguous")
    if rows <= 1 or cols == 0:
        return cols if cols > 1 else 1
    if s0 < cols:
        raise ValueError(f"{name} rows must not overlap; an expanded tensor needs .contiguous()")
    return s0


def _matrix(t, name, device, rows=None, cols=None):
    """(pointer, pitch, rows, cols) of a 2-D float32 tensor on ``device``, of
    the given sizes where they are given."""
    import torch
    if t.dtype is not torch.float32 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must be {'?' if rows is None else rows}x"
                         f"{'?' if cols is None else cols}, got {r}x{c}")
    s0, s1 = t.stride()
    return t.data_ptr(), _rows(r, c, s0, s1, name), r, c


def _stack(t, name, device, groups, rows=None, cols=None):
    """(pointer, pitch, stride, rows, cols) of a 3-D float32 tensor on
    ``device``: one matrix per group, of the given sizes where they are given."""
    import torch
    if t.dtype is not torch.float32 or t.dim() != 3:
        raise TypeError(f"{name} must be a 3-D float32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    g, r, c = t.shape
    if g != groups or (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must be {groups}x{'?' if rows is None else rows}x"
                         f"{'?' if cols is None else cols}, got {g}x{r}x{c}")
    sg, s0, s1 = t.stride()
    return t.data_ptr(), _rows(r, c, s0, s1, name), sg, r, c


def _vector(t, name, device, count):
    """Pointer of a contiguous float32 vector on ``device`` (0 for None)."""
    import torch
    if t is None:
        return 0
    if (t.dtype is not torch.float32 or t.dim() != 1 or t.shape[0] != count
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous vector of {count} floats")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    return t.data_ptr()


def _biases(t, device, groups, cols):
    """(pointer, stride) of one bias row per group; (0, 0) for None."""
    import torch
    if t is None:
        return 0, 0
    if t.dtype is not torch.float32 or tuple(t.shape) != (groups, cols):
        raise ValueError(f"bias must be {groups}x{cols} floats, got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("bias rows must be contiguous")
    if t.device != device:
        raise ValueError(f"bias must be on {device} (got {t.device})")
    return t.data_ptr(), t.stride(0)


def _gpu(t, name):
    if t.device.type != "cuda":
        raise TypeError(f"{name} must be on a GPU (got {t.device})")
    return t.device


def _groups_of(offsets):
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold one entry more than there are groups")
    return offsets.shape[0] - 1


def group_rows(index, groups, *, per_row=1):
    """The entries of a 1-D int32 GPU tensor ordered by the group they name
    (values outside [0, groups) name none).  Returns int32 tensors ``offsets``
    (groups + 1), ``order`` (the entries by (group, entry)) and ``rows``
    (order // per_row); both hold -1 from offsets[groups] on.  (The three are
    parts of one allocation.)"""
    dev = _gpu(index, "index")
    ptr = _index(index, "index", dev)
    n, groups = index.shape[0], int(groups)
    places = max(groups, 0) + 1
    offsets, order, rows = index.new_empty(places + 2 * n).split_with_sizes((places, n, n))
    rc = _on(index, gemm_f32_group_rows, n, groups, int(per_row), ptr, offsets.data_ptr(),
             order.data_ptr(), rows.data_ptr())
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_group_rows")
    return offsets, order, rows


def gemm_grouped(A, B, offsets, C=None, *, trans_b=False, alpha=1.0, beta=0.0, bias=None,
                 act=ACT_NONE, index_a=None, index_c=None):
    """C[index_c[i]] = act(alpha * A[index_a[i]] @ op(B[g]) + beta * C[index_c[i]]
    + bias[g]) for every place i of group g (offsets[g] <= i < offsets[g + 1]).
    B is groups x K x N (groups x N x K when trans_b), bias groups x N or None;
    an index that is None is the identity.  The places are the indexes' length
    (A's rows without any).  A new C has one row a place; rows that no place
    names hold nothing in particular there, and keep what they held in a C that
    is given.  Returns C."""
    dev, groups = _gpu(A, "A"), _groups_of(offsets)
    a, lda, rows_a, K = _matrix(A, "A", dev)
    b, ldb, sb, b_rows, b_cols = _stack(B, "B", dev, groups, *((None, K) if trans_b else (K,)))
    N = b_rows if trans_b else b_cols
    rows = (index_a.shape[0] if index_a is not None else
            index_c.shape[0] if index_c is not None else rows_a)
    ia, ic = _index(index_a, "index_a", dev, rows), _index(index_c, "index_c", dev, rows)
    if C is None:
        C = A.new_empty((rows, N))
    c, ldc, rows_c, _ = _matrix(C, "C", dev, cols=N)
    bptr, sbias = _biases(bias, dev, groups, N)
    rc = _on(A, gemm_f32_grouped, 1 if trans_b else 0, rows, N, K, groups,
             _index(offsets, "offsets", dev), alpha, a, lda, rows_a, ia, b, ldb, sb, beta, c, ldc,
             rows_c, ic, bptr, sbias, int(act))
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_grouped")
    return C


def gemm_grouped_wgrad(A, B, offsets, C=None, *, alpha=1.0, beta=0.0, index_a=None,
                       index_b=None):
    """C[g] = alpha * sum over the places i of group g of A[index_a[i]]^T
    B[index_b[i]], plus beta * C[g]: the gradient of gemm_grouped's weights.
    Returns C (groups x A's columns x B's columns)."""
    dev, groups = _gpu(A, "A"), _groups_of(offsets)
    a, lda, rows_a, M = _matrix(A, "A", dev)
    b, ldb, rows_b, N = _matrix(B, "B", dev)
    rows = (index_a.shape[0] if index_a is not None else
            index_b.shape[0] if index_b is not None else rows_a)
    ia, ib = _index(index_a, "index_a", dev, rows), _index(index_b, "index_b", dev, rows)
    if C is None:
        C = A.new_empty((groups, M, N))
    c, ldc, sc, _, _ = _stack(C, "C", dev, groups, M, N)
    rc = _on(A, gemm_f32_grouped_wgrad, rows, M, N, groups, _index(offsets, "offsets", dev), alpha,
             a, lda, rows_a, ia, b, ldb, rows_b, ib, beta, c, ldc, sc)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_grouped_wgrad")
    return C


def gemm_adapters(X, W, down, up, offsets, order, Y=None, H=None, *, trans=False, scale=None,
                  bias=None):
    """Y = X @ op(W) + bias, and for the rows order[i] of adapter g
    (offsets[g] <= i < offsets[g + 1]) H[i] = scale[g] * X[order[i]] @ op(down[g]),
    Y[order[i]] += H[i] @ op(up[g]).  W is K x N, down adapters x K x R and up
    adapters x R x N, or with ``trans`` each matrix stored transposed; ``scale``
    one float per adapter (None: 1), ``bias`` N floats or None.  Returns (Y, H);
    H (one row a place) is what gemm_adapters_grad takes."""
    dev, adapters = _gpu(X, "X"), _groups_of(offsets)
    x, ldx, M, K = _matrix(X, "X", dev)
    w, ldw, w_rows, w_cols = _matrix(W, "W", dev, *((None, K) if trans else (K,)))
    d, ldd, sd, d_rows, d_cols = _stack(down, "down", dev, adapters,
                                        *((None, K) if trans else (K,)))
    N, R = (w_rows, d_rows) if trans else (w_cols, d_cols)
    u, ldu, su, _, _ = _stack(up, "up", dev, adapters, *((N, R) if trans else (R, N)))
    places = order.shape[0]
    if Y is None:
        Y = X.new_empty((M, N))
    if H is None:
        H = X.new_empty((places, R))
    y, ldy, _, _ = _matrix(Y, "Y", dev, M, N)
    h, ldh, _, _ = _matrix(H, "H", dev, places, R)
    rc = _on(X, gemm_f32_adapters, 1 if trans else 0, M, N, K, R, adapters, places,
             _index(offsets, "offsets", dev), _index(order, "order", dev),
             _vector(scale, "scale", dev, adapters), x, ldx, w, ldw, d, ldd, sd, u, ldu, su,
             _vector(bias, "bias", dev, N), h, ldh, y, ldy)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_adapters")
    return Y, H


def gemm_adapters_grad(dY, X, W, down, up, offsets, order, H, *, trans=False, scale=None):
    """Gradients of gemm_adapters with the H it returned: (dX, d_down, d_up) for
    the gradient dY of Y.  (W's is gemm_ex's product of X and dY, the bias's the
    sum of dY's rows.)"""
    dX, G = gemm_adapters(dY, W, up, down, offsets, order, trans=not trans, scale=scale)
    if trans:
        return (dX, gemm_grouped_wgrad(G, X, offsets, index_b=order),
                gemm_grouped_wgrad(dY, H, offsets, index_a=order))
    return (dX, gemm_grouped_wgrad(X, G, offsets, index_a=order),
            gemm_grouped_wgrad(H, dY, offsets, index_b=order))


# ---- around an expert layer ----------------------------------------------------

def _entries(t, name, dtype, device, rows, cols):
    """Pointer of a contiguous rows x cols tensor on ``device`` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or tuple(t.shape) != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {rows}x{cols} {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    return t.data_ptr()


def route(logits, top, *, bias=None, score=SCORE_SOFTMAX, groups=1, group_top=None, group_best=1,
          renorm=False, scale=1.0):
    """The ``top`` experts of each row of ``logits`` (tokens x experts) by softmax
    or sigmoid scores plus ``bias`` (experts floats or None), and their weights:
    scale * score, over the sum of the token's chosen scores with ``renorm``.  With
    ``groups`` of experts only those of the ``group_top`` best groups are taken, a
    group's score being its best value or the sum of its best ``group_best`` = 2.
    Returns (choice, weight), tokens x top: int32 with -1 (and weight 0) where too
    few experts are left, as group_rows takes them, and float32."""
    import torch
    dev = _gpu(logits, "logits")
    ptr, ldl, tokens, experts = _matrix(logits, "logits", dev)
    top, groups = int(top), int(groups)
    choice = logits.new_empty((tokens, max(top, 0)), dtype=torch.int32)
    weight = logits.new_empty((tokens, max(top, 0)))
    rc = _on(logits, gemm_f32_route, tokens, experts, top, ptr, ldl,
             _vector(bias, "bias", dev, experts), int(score), groups,
             groups if group_top is None else int(group_top), int(group_best), 1 if renorm else 0,
             scale, choice.data_ptr(), weight.data_ptr())
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_route")
    return choice, weight


def route_grad(dweight, logits, choice, *, score=SCORE_SOFTMAX, renorm=False, scale=1.0,
               dlogits=None):
    """Gradient of route's weights with respect to the logits, from the weights'
    (tokens x top) and the choices that route returned.  Returns dlogits."""
    import torch
    dev = _gpu(logits, "logits")
    ptr, ldl, tokens, experts = _matrix(logits, "logits", dev)
    if choice.dim() != 2:
        raise ValueError("choice must be tokens x top")
    top = choice.shape[1]
    c = _entries(choice, "choice", torch.int32, dev, tokens, top)
    dw = _entries(dweight, "dweight", torch.float32, dev, tokens, top)
    if dlogits is None:
        dlogits = logits.new_empty((tokens, experts))
    d, ldd, _, _ = _matrix(dlogits, "dlogits", dev, tokens, experts)
    rc = _on(logits, gemm_f32_route_grad, tokens, experts, top, ptr, ldl, int(score),
             1 if renorm else 0, scale, c, dw, d, ldd)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_route_grad")
    return dlogits


def join_rows(H, weight, choice=None, Y=None, *, groups=MAX_GROUPS, beta=0.0):
    """Y[t] = sum over j of weight[t, j] * H[t * top + j], plus beta * Y[t]: the
    experts' rows of each token added up.  Entries whose choice (int32, tokens x
    top; None: all count) is outside [0, groups) are left out.  Returns Y."""
    import torch
    dev = _gpu(H, "H")
    if weight.dim() != 2:
        raise ValueError("weight must be tokens x top")
    tokens, top = weight.shape
    h, ldh, _, N = _matrix(H, "H", dev, tokens * top)
    w = _entries(weight, "weight", torch.float32, dev, tokens, top)
    c = _entries(choice, "choice", torch.int32, dev, tokens, top)
    if Y is None:
        Y = H.new_empty((tokens, N))
    y, ldy, _, _ = _matrix(Y, "Y", dev, tokens, N)
    rc = _on(H, gemm_f32_join_rows, tokens, top, N, h, ldh, w, c, int(groups), beta, y, ldy)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_join_rows")
    return Y


def join_rows_grad(dY, H, weight, choice=None, dH=None, *, groups=MAX_GROUPS):
    """Gradients of join_rows for the gradient dY of Y: (dH, dweight), zeros at the
    entries that are left out."""
    import torch
    dev = _gpu(H, "H")
    if weight.dim() != 2:
        raise ValueError("weight must be tokens x top")
    tokens, top = weight.shape
    h, ldh, _, N = _matrix(H, "H", dev, tokens * top)
    dy, lddy, _, _ = _matrix(dY, "dY", dev, tokens, N)
    w = _entries(weight, "weight", torch.float32, dev, tokens, top)
    c = _entries(choice, "choice", torch.int32, dev, tokens, top)
    if dH is None:
        dH = H.new_empty((tokens * top, N))
    d, lddh, _, _ = _matrix(dH, "dH", dev, tokens * top, N)
    dweight = H.new_empty((tokens, top))
    rc = _on(H, gemm_f32_join_rows_grad, tokens, top, N, dy, lddy, h, ldh, w, c, int(groups), d,
             lddh, dweight.data_ptr())
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_join_rows_grad")
    return dH, dweight


def _scale_type(t):
    import torch
    types = {torch.float32: SCALE_F32, torch.float16: SCALE_F16, torch.bfloat16: SCALE_BF16,
             torch.uint8: SCALE_E8M0, torch.float8_e8m0fnu: SCALE_E8M0}
    if t.dtype not in types:
        raise TypeError(f"scale must be float32, float16, bfloat16 or e8m0 bytes, not {t.dtype}")
    return types[t.dtype]


def _packed(t, name, device, lead, rows, cols):
    """(pointer, pitch, stride) of a tensor lead + (rows, cols) on ``device`` whose
    rows are contiguous, in elements; lead is () or (groups,)."""
    if tuple(t.shape) != (*lead, rows, cols):
        raise ValueError(f"{name} must be {'x'.join(map(str, (*lead, rows, cols)))}, got "
                         f"{'x'.join(map(str, t.shape))}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    s = t.stride()
    return t.data_ptr(), _rows(rows, cols, s[-2], s[-1], name), s[0] if lead else 0


def _q4(codes, scale, zero, group, format, device, lead, K):
    """The arguments of 4-bit weights, N x K (for each of lead): (N, format ... ldz)
    and the three strides."""
    import torch
    if codes.dtype is not torch.uint8 or codes.dim() != len(lead) + 2:
        raise TypeError(f"codes must be a {len(lead) + 2}-D uint8 tensor")
    group = int(group)
    if group < 1:
        raise ValueError("group must be positive")
    N, along = codes.shape[-2], (K + group - 1) // group
    q, ldq, sq = _packed(codes, "codes", device, lead, N, (K + 1) // 2)
    kind = _scale_type(scale)
    s, lds, ss = _packed(scale, "scale", device, lead, N, along)
    z, ldz, sz = 0, 1, 0
    if zero is not None:
        if zero.dtype is not torch.uint8:
            raise TypeError("zero must be a uint8 tensor")
        z, ldz, sz = _packed(zero, "zero", device, lead, N, along)
    return N, int(format), group, q, ldq, sq, kind, s, lds, ss, z, ldz, sz


def gemm_q4(A, codes, scale, C=None, *, zero=None, group=128, format=Q4_INT, alpha=1.0, beta=0.0,
            bias=None, act=ACT_NONE):
    """C = act(alpha * A @ W.T + beta * C + bias) with W (N x K) in 4 bits: ``codes``
    uint8, N x (K + 1) // 2, the even k in a byte's low half; ``scale`` N x groups of
    K, float32, float16, bfloat16 or e8m0 bytes; Q4_INT: (code - zero) * scale with
    ``zero`` uint8 like scale (None: 8), Q4_E2M1: the e2m1 value * scale.  ``group`` is
    a power of two from 32 on.  (q4.quantize makes them from a matrix.)  Returns C."""
    dev = _gpu(A, "A")
    a, lda, M, K = _matrix(A, "A", dev)
    N, fmt, group, q, ldq, _, kind, s, lds, _, z, ldz, _ = _q4(codes, scale, zero, group, format,
                                                               dev, (), K)
    if C is None:
        C = A.new_empty((M, N))
    c, ldc, _, _ = _matrix(C, "C", dev, M, N)
    rc = _on(A, gemm_f32_q4, M, N, K, alpha, a, lda, fmt, group, q, ldq, kind, s, lds, z, ldz,
             beta, c, ldc, _vector(bias, "bias", dev, N), int(act))
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_q4")
    return C


def gemm_q4_grouped(A, codes, scale, offsets, C=None, *, zero=None, group=128, format=Q4_INT,
                    alpha=1.0, beta=0.0, bias=None, act=ACT_NONE, index_a=None, index_c=None):
    """gemm_grouped with weights in 4 bits: C[index_c[i]] = act(alpha * A[index_a[i]]
    @ W[g].T + beta * C[index_c[i]] + bias[g]) for every place i of group g, with
    ``codes``, ``scale`` and ``zero`` as gemm_q4 takes them, one matrix for each group.
    Returns C."""
    dev, groups = _gpu(A, "A"), _groups_of(offsets)
    a, lda, rows_a, K = _matrix(A, "A", dev)
    N, fmt, group, q, ldq, sq, kind, s, lds, ss, z, ldz, sz = _q4(codes, scale, zero, group, format,
                                                                  dev, (groups,), K)
    rows = (index_a.shape[0] if index_a is not None else
            index_c.shape[0] if index_c is not None else rows_a)
    ia, ic = _index(index_a, "index_a", dev, rows), _index(index_c, "index_c", dev, rows)
    if C is None:
        C = A.new_empty((rows, N))
    c, ldc, rows_c, _ = _matrix(C, "C", dev, cols=N)
    bptr, sbias = _biases(bias, dev, groups, N)
    rc = _on(A, gemm_f32_q4_grouped, rows, N, K, groups, _index(offsets, "offsets", dev), alpha, a,
             lda, rows_a, ia, fmt, group, q, ldq, sq, kind, s, lds, ss, z, ldz, sz, beta, c, ldc,
             rows_c, ic, bptr, sbias, int(act))
    if rc != GEMM_F32_OK:
        raise GemmError(rc, "gemm_f32_q4_grouped")
    return C


def _arrays(tensors, name, device):
    """Host tables of the pointers and sizes of contiguous float32 tensors.  (There may
    be hundreds: each property is read by one map, without a Python frame for each.)"""
    import torch
    T = torch.Tensor
    for t in set(map(type, tensors)):
        if not issubclass(t, T):
            raise TypeError(f"{name} must hold tensors")
    if set(map(T.get_device, tensors)) != {device.index}:
        raise ValueError(f"{name} must be on {device}")
    if (set(map(T.dtype.__get__, tensors)) != {torch.float32}
            or not all(map(T.is_contiguous, tensors))):
        raise TypeError(f"{name} must hold contiguous float32 tensors")
    return (array("Q", map(T.data_ptr, tensors)), array("q", map(T.numel, tensors)))


def _norm_of(tensors, out, max_norm, norm):
    import torch
    tensors = list(tensors)
    if not tensors:
        raise ValueError("there are no tensors")
    dev = _gpu(tensors[0], "tensors")
    x, n = _arrays(tensors, "tensors", dev)
    y = None
    if out is not None:
        out = list(out)
        y, m = _arrays(out, "out", dev)
        if m != n:
            raise ValueError("out must hold a tensor of the same size for each")
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    ptr = _vector(norm, "norm", dev, 1)
    if max_norm is None:
        rc, what = (_on(tensors[0], gemm_f32_norm, len(tensors), x.buffer_info()[0],
                        n.buffer_info()[0], ptr), "gemm_f32_norm")
    else:
        rc, what = (_on(tensors[0], gemm_f32_clip, len(tensors), x.buffer_info()[0],
                        n.buffer_info()[0], y and y.buffer_info()[0], max_norm, ptr),
                    "gemm_f32_clip")
    if rc != GEMM_F32_OK:
        raise GemmError(rc, what)
    return norm


def norm(tensors, norm=None):
    """The norm of all elements of contiguous float32 GPU tensors (a model's
    gradients) together, as a 1-element tensor, summed in 64 bits."""
    return _norm_of(tensors, None, None, norm)


def clip_norm(tensors, max_norm, out=None, norm=None):
    """The tensors scaled by max_norm / norm where their norm together is above
    max_norm: in place, or into the tensors of ``out``.  A norm that is not finite
    leaves them as they are.  Returns the norm before, a 1-element tensor."""
    if max_norm is None:
        raise TypeError("max_norm must be a number")
    return _norm_of(tensors, out, max_norm, norm)


class _device:
    """Make the tensor's device current for the call (the library uses the
    current HIP device)."""

    def __init__(self, t):
        self.idx = t.device.index

    def __enter__(self):
        import torch
        self.prev = torch.cuda.current_device()
        if self.idx is not None and self.idx != self.prev:
            torch.cuda.set_device(self.idx)

    def __exit__(self, *exc):
        import torch
        if self.idx is not None and self.idx != self.prev:
            torch.cuda.set_device(self.prev)
        return False
