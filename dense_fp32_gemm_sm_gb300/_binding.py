"""Binding of the C ABI declared in ``include/fgemm.h``: ctypes, and a small C module for the
MXFP4 and 16-bit calls.

Argument marshalling only: every call goes straight to ``libfgemm.so`` and the
work runs in its CUDA kernels.  Matrices may be given as CUDA float32 torch
tensors (their ``data_ptr()`` is passed) or as raw device addresses (ints).
When no stream is given and a tensor is passed, torch's current stream on that
tensor's device is used; otherwise the legacy default stream (0).

There is no CPU fallback: if the library cannot be built or loaded, every call
raises.
"""

from __future__ import annotations

import ctypes
import sys
import threading

from . import _build

OP_N, OP_T = 0, 1
OK, ERR_INVALID_VALUE, ERR_LAUNCH, ERR_NOT_SUPPORTED, ERR_TIMEOUT = 0, 1, 2, 3, 4
MATH_FP32, MATH_TF32, MATH_3XTF32 = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = 0, 1, 2, 3
MAX_GROUPS = 1024  # FGEMM_MAX_GROUPS of include/fgemm.h

_lock = threading.Lock()
_lib = None

_c_int, _c_float, _c_ll, _c_vp = ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_void_p


class FgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def library() -> ctypes.CDLL:
    """Load (building first if the sources are newer) ``libfgemm.so``."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            lib = ctypes.CDLL(path)
            sig = {
                "fgemm_sgemm": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _c_vp, _c_int,
                                _c_vp, _c_int, _c_float, _c_vp, _c_int, _c_vp],
                "fgemm_sgemm_bias_relu": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _c_vp,
                                          _c_int, _c_vp, _c_int, _c_float, _c_vp, _c_int, _c_vp,
                                          _c_int, _c_vp],
                "fgemm_sgemm_row_bias_relu": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                              _c_vp, _c_int, _c_vp, _c_int, _c_float, _c_vp,
                                              _c_int, _c_vp, _c_int, _c_vp],
                "fgemm_sgemm_strided_batched": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                                _c_vp, _c_int, _c_ll, _c_vp, _c_int, _c_ll,
                                                _c_float, _c_vp, _c_int, _c_ll, _c_int, _c_vp],
                "fgemm_gemm_explicit": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                        _c_vp, _c_int, _c_ll, _c_vp, _c_int, _c_ll, _c_float,
                                        _c_vp, _c_int, _c_ll, _c_int, _c_vp, _c_int, _c_vp],
                "fgemm_gemm_math": [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                    _c_vp, _c_int, _c_ll, _c_vp, _c_int, _c_ll, _c_float,
                                    _c_vp, _c_int, _c_ll, _c_int, _c_vp, _c_int, _c_vp],
                "fgemm_device_status": [_c_int],
                "fgemm_select_config": [_c_int] * 8,
                "fgemm_launch_count": [_c_int] * 9,
                "fgemm_num_configs": [],
                "fgemm_config_name": [_c_int],
                "fgemm_status_string": [_c_int],
            }
            for name, argtypes in sig.items():
                fn = getattr(lib, name)
                fn.argtypes = argtypes
                fn.restype = _c_int
            lib.fgemm_sgemm_splitk.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                               _c_vp, _c_int, _c_vp, _c_int, _c_float, _c_vp,
                                               _c_int, _c_vp, _c_int, _c_int, _c_vp,
                                               ctypes.c_size_t, _c_vp]
            lib.fgemm_sgemm_splitk.restype = _c_int
            lib.fgemm_sgemm_splitk_noalloc.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int,
                                                       _c_float, _c_vp, _c_int, _c_vp, _c_int,
                                                       _c_float, _c_vp, _c_int, _c_vp, _c_int,
                                                       _c_int, _c_vp]
            lib.fgemm_sgemm_splitk_noalloc.restype = _c_int
            lib.fgemm_splitk_workspace_size.argtypes = [_c_int, _c_int, _c_int, _c_int]
            lib.fgemm_splitk_workspace_size.restype = ctypes.c_size_t
            lib.fgemm_staged_workspace_size.argtypes = [_c_int] * 6
            lib.fgemm_staged_workspace_size.restype = ctypes.c_size_t
            lib.fgemm_staged_choice.argtypes = [_c_int] * 10 + [ctypes.c_size_t, _c_int]
            lib.fgemm_staged_choice.restype = _c_int
            lib.fgemm_sgemm_staged.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                               _c_vp, _c_int, _c_ll, _c_vp, _c_int, _c_ll,
                                               _c_float, _c_vp, _c_int, _c_ll, _c_int, _c_vp,
                                               _c_int, _c_int, _c_vp, ctypes.c_size_t, _c_vp]
            lib.fgemm_sgemm_staged.restype = _c_int
            lib.fgemm_math_staged_workspace_size.argtypes = [_c_int] * 7
            lib.fgemm_math_staged_workspace_size.restype = ctypes.c_size_t
            lib.fgemm_math_staged_choice.argtypes = [_c_int] * 11 + [ctypes.c_size_t, _c_int]
            lib.fgemm_math_staged_choice.restype = _c_int
            lib.fgemm_gemm_math_staged.argtypes = [_c_int] + lib.fgemm_sgemm_staged.argtypes
            lib.fgemm_gemm_math_staged.restype = _c_int
            lib.fgemm_math_supported.argtypes = [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                                 _c_float, _c_vp, _c_int, _c_ll, _c_vp, _c_int,
                                                 _c_ll, _c_int]
            lib.fgemm_math_supported.restype = _c_int
            lib.fgemm_debug_withhold_tensor_core.argtypes = [_c_int, _c_ll]
            lib.fgemm_debug_withhold_tensor_core.restype = None
            _sz = ctypes.c_size_t
            for name, argtypes, restype in (
                    ("codes_size", [_c_int] * 2, _sz),
                    ("scales_size", [_c_int] * 2, _sz),
                    ("quantize_grad_workspace_size", [_c_int] * 2, _sz),
                    ("plan", [_c_int] * 5, _c_int),
                    ("linear_workspace_size", [_c_int] * 3, _sz)):
                fn = getattr(lib, "fgemm_mxfp4_" + name)
                fn.argtypes = argtypes
                fn.restype = restype
            for name, argtypes, restype in (
                    ("copy_workspace_size", [_c_int] * 6, _sz),
                    ("sums_workspace_size", [_c_int] * 3, _sz),
                    ("plan", [_c_int] * 8, _c_int)):
                fn = getattr(lib, "fgemm_gemm16_" + name)
                fn.argtypes = argtypes
                fn.restype = restype
            lib.fgemm_config_name.restype = ctypes.c_char_p
            lib.fgemm_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    if hasattr(x, "data_ptr"):
        if x.numel() and (not x.is_cuda or x.dtype.itemsize != 4 or not x.is_floating_point()):
            raise TypeError("fgemm takes CUDA float32 tensors (got %s on %s)" % (x.dtype, x.device))
        return x.data_ptr() or None
    raise TypeError("expected a CUDA tensor or a device address, got %r" % type(x))


def _stream(stream, *tensors):
    if stream is None:
        for t in tensors:
            if hasattr(t, "is_cuda") and t.is_cuda:
                import torch
                return torch.cuda.current_stream(t.device).cuda_stream
        return None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream  # a torch.cuda.Stream


def _check(status: int, where: str):
    if status != OK:
        raise FgemmError(status, where)


def status_string(status: int) -> str:
    return library().fgemm_status_string(int(status)).decode()


def num_configs() -> int:
    return library().fgemm_num_configs()


def config_name(config: int):
    name = library().fgemm_config_name(int(config))
    return name.decode() if name else None


def select_config(transa, transb, M, N, K, batch, aligned, num_sms) -> int:
    return library().fgemm_select_config(int(transa), int(transb), M, N, K, batch,
                                         1 if aligned else 0, num_sms)


def launch_count(config, transa, transb, M, N, K, batch, aligned, num_sms) -> int:
    """``fgemm_launch_count``: kernel launches of one call (config < 0: as selected)."""
    return library().fgemm_launch_count(int(config), int(transa), int(transb), M, N, K, batch,
                                        1 if aligned else 0, num_sms)


def sgemm(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None,
          check=True) -> int:
    """``fgemm_sgemm``: C = alpha*op(A)*op(B) + beta*C (row-major, see include/fgemm.h)."""
    st = library().fgemm_sgemm(int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, _ptr(B),
                               ldb, beta, _ptr(C), ldc, _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm")
    return st


def sgemm_bias_relu(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias,
                    apply_relu, stream=None, check=True) -> int:
    """``fgemm_sgemm_bias_relu``: C = relu?(alpha*op(A)*op(B) + beta*C + bias[col])."""
    st = library().fgemm_sgemm_bias_relu(int(transa), int(transb), M, N, K, alpha, _ptr(A), lda,
                                         _ptr(B), ldb, beta, _ptr(C), ldc, _ptr(bias),
                                         1 if apply_relu else 0, _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_bias_relu")
    return st


def sgemm_row_bias_relu(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, row_bias,
                        apply_relu, stream=None, check=True) -> int:
    """``fgemm_sgemm_row_bias_relu``: C = relu?(alpha*op(A)*op(B) + beta*C + row_bias[row])."""
    st = library().fgemm_sgemm_row_bias_relu(int(transa), int(transb), M, N, K, alpha, _ptr(A),
                                             lda, _ptr(B), ldb, beta, _ptr(C), ldc, _ptr(row_bias),
                                             1 if apply_relu else 0, _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_row_bias_relu")
    return st


def sgemm_strided_batched(transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta,
                          C, ldc, strideC, batch, stream=None, check=True) -> int:
    """``fgemm_sgemm_strided_batched``: the plain GEMM on batch offsets b*stride."""
    st = library().fgemm_sgemm_strided_batched(
        int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb, strideB,
        beta, _ptr(C), ldc, strideC, batch, _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_strided_batched")
    return st


def gemm_explicit(config, transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta,
                  C, ldc, strideC, batch, bias=None, apply_relu=False, stream=None,
                  check=True) -> int:
    """``fgemm_gemm_explicit``: every option, with an explicit kernel configuration."""
    st = library().fgemm_gemm_explicit(
        int(config), int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb,
        strideB, beta, _ptr(C), ldc, strideC, batch, _ptr(bias), 1 if apply_relu else 0,
        _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_gemm_explicit")
    return st


def gemm_math(math, transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C,
              ldc, strideC, batch, bias=None, apply_relu=False, stream=None, check=True) -> int:
    """``fgemm_gemm_math``: FP32 CUDA cores (MATH_FP32) or tcgen05 TF32 / 3xTF32."""
    st = library().fgemm_gemm_math(
        int(math), int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb,
        strideB, beta, _ptr(C), ldc, strideC, batch, _ptr(bias), 1 if apply_relu else 0,
        _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_gemm_math")
    return st


def math_supported(math, transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB,
                   batch) -> int:
    """``fgemm_math_supported``: 1 if ``gemm_math`` runs the requested arithmetic for these
    operands, 0 if it would use the FP32 CUDA-core kernel instead, -1 for a bad ``math``.
    Host-only; the pointers are only tested for alignment."""
    return library().fgemm_math_supported(int(math), int(transa), int(transb), M, N, K, alpha,
                                          _ptr(A), lda, strideA, _ptr(B), ldb, strideB, batch)


def device_status(clear=True) -> int:
    """``fgemm_device_status``: ERR_TIMEOUT if a tensor-core wait ran out (call after a sync)."""
    return library().fgemm_device_status(1 if clear else 0)


def debug_withhold_tensor_core(k_block: int, wait_limit_ns: int = 0) -> None:
    """Testing: ``fgemm_debug_withhold_tensor_core`` (k_block < 0 restores normal runs)."""
    library().fgemm_debug_withhold_tensor_core(int(k_block), int(wait_limit_ns))


def splitk_workspace_size(M, N, K, splits) -> int:
    """``fgemm_splitk_workspace_size``: bytes of workspace fgemm_sgemm_splitk needs (0: invalid)."""
    return int(library().fgemm_splitk_workspace_size(M, N, K, splits))


def sgemm_splitk(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, apply_relu,
                 splits, workspace, workspace_bytes, stream=None, check=True) -> int:
    """``fgemm_sgemm_splitk``: split-K GEMM with a caller-owned workspace."""
    st = library().fgemm_sgemm_splitk(
        int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
        _ptr(bias), 1 if apply_relu else 0, int(splits), _ptr(workspace), int(workspace_bytes),
        _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_splitk")
    return st


# FGEMM_MAX_DIM of include/fgemm.h: the largest M, N or K a call takes (2^31 - 256);
# larger sizes return FGEMM_ERR_NOT_SUPPORTED.
MAX_DIM = 2**31 - 256


# FGEMM_NOALLOC_SCRATCH_BYTES of include/fgemm.h: the fixed scratch array behind
# fgemm_sgemm_splitk_noalloc.
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def sgemm_splitk_noalloc(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias,
                         apply_relu, splits, stream=None, check=True) -> int:
    """``fgemm_sgemm_splitk_noalloc``: split-K GEMM whose partial products live in the
    library's fixed device array instead of a caller workspace (for callers that may
    not allocate device memory)."""
    st = library().fgemm_sgemm_splitk_noalloc(
        int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
        _ptr(bias), 1 if apply_relu else 0, int(splits), _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_splitk_noalloc")
    return st


# stage = -1 for fgemm_sgemm_staged: the launch-time model chooses.
STAGE_AUTO = -1


def staged_workspace_size(transa, transb, M, N, K, batch) -> int:
    """``fgemm_staged_workspace_size``: bytes of workspace fgemm_sgemm_staged needs."""
    return int(library().fgemm_staged_workspace_size(int(transa), int(transb), M, N, K, batch))


def staged_choice(transa, transb, M, N, K, batch, shared_a, shared_b, aligned_a, aligned_b,
                  num_sms, workspace_bytes=None) -> int:
    """``fgemm_staged_choice``: which operands a staged call copies into its workspace
    (bit 0: A, bit 1: B) by the launch-time model; host-only.  workspace_bytes=None:
    the full fgemm_staged_workspace_size."""
    if workspace_bytes is None:
        workspace_bytes = staged_workspace_size(transa, transb, M, N, K, max(1, batch))
    return library().fgemm_staged_choice(int(transa), int(transb), M, N, K, batch,
                                         1 if shared_a else 0, 1 if shared_b else 0,
                                         1 if aligned_a else 0, 1 if aligned_b else 0,
                                         int(workspace_bytes), num_sms)


def sgemm_staged(transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                 strideC, batch, bias, apply_relu, stage, workspace, workspace_bytes,
                 stream=None, check=True) -> int:
    """``fgemm_sgemm_staged``: the GEMM after copying operands into a caller workspace
    (transposed k-major, or re-pitched when unaligned; stage = STAGE_AUTO: the copies the
    model finds faster among those that fit)."""
    st = library().fgemm_sgemm_staged(
        int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb, strideB,
        beta, _ptr(C), ldc, strideC, batch, _ptr(bias), 1 if apply_relu else 0, int(stage),
        _ptr(workspace), int(workspace_bytes), _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_sgemm_staged")
    return st


def math_staged_workspace_size(math, transa, transb, M, N, K, batch) -> int:
    """``fgemm_math_staged_workspace_size``: bytes of workspace fgemm_gemm_math_staged needs
    for both copies."""
    return int(library().fgemm_math_staged_workspace_size(int(math), int(transa), int(transb), M,
                                                          N, K, batch))


def math_staged_choice(math, transa, transb, M, N, K, batch, shared_a, shared_b, aligned_a,
                       aligned_b, num_sms, workspace_bytes=None) -> int:
    """``fgemm_math_staged_choice``: the copies fgemm_gemm_math_staged makes with
    stage = STAGE_AUTO (bit 0: A, bit 1: B); host-only.  workspace_bytes=None: the full
    fgemm_math_staged_workspace_size."""
    if workspace_bytes is None:
        workspace_bytes = math_staged_workspace_size(math, transa, transb, M, N, K, max(1, batch))
    return library().fgemm_math_staged_choice(int(math), int(transa), int(transb), M, N, K, batch,
                                              1 if shared_a else 0, 1 if shared_b else 0,
                                              1 if aligned_a else 0, 1 if aligned_b else 0,
                                              int(workspace_bytes), num_sms)


def gemm_math_staged(math, transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB,
                     beta, C, ldc, strideC, batch, bias, apply_relu, stage, workspace,
                     workspace_bytes, stream=None, check=True) -> int:
    """``fgemm_gemm_math_staged``: fgemm_gemm_math after copying operands K-major into a
    caller workspace (stage = STAGE_AUTO: the library's choice among the copies that fit)."""
    st = library().fgemm_gemm_math_staged(
        int(math), int(transa), int(transb), M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb,
        strideB, beta, _ptr(C), ldc, strideC, batch, _ptr(bias), 1 if apply_relu else 0,
        int(stage), _ptr(workspace), int(workspace_bytes), _stream(stream, C, A, B))
    if check:
        _check(st, "fgemm_gemm_math_staged")
    return st


# ---- MXFP4 (see "MXFP4" in include/fgemm.h) -------------------------------------------

# The calls' arguments are converted by a small C module (csrc/py_calls.c); it takes tensors or
# addresses like the functions above.  Tensors have to be on the current device (ValueError): the
# library launches there.

_TYPE_NAMES = ("torch.float32", "torch.bfloat16", "torch.float16", "torch.int32")
_calls = None


def _type_of(dtype):
    """fgemm_dtype value of a torch dtype (this module does not import torch), 3 for int32, or -1."""
    name = str(dtype)
    return _TYPE_NAMES.index(name) if name in _TYPE_NAMES else -1


def _current_stream(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _current_device():
    import torch
    return torch.cuda.current_device()


def _native():
    """Load the C module (building first if its source is newer) and give it the library's entries."""
    global _calls
    lib = library()
    with _lock:
        if _calls is None:
            _build.build_calls()
            from . import _calls as module
            raw_stream, device, one_device = _current_stream, _current_device, False
            if "torch" in sys.modules:
                try:  # the handle without a Stream object, which takes 2 us
                    from torch._C import _cuda_getCurrentRawStream as raw_stream, _cuda_getDevice as device
                except ImportError:
                    pass
                # Where torch sees one device, the calls need not ask which one is current (0.4 us).
                one_device = sys.modules["torch"].cuda.device_count() == 1
            module.bind(_type_of, raw_stream, device, one_device,
                        *(ctypes.cast(getattr(lib, "fgemm_" + name), _c_vp).value
                          for name in ("mxfp4_quantize", "mxfp4_quantize_grad", "mxfp4_dequantize", "mxfp4_gemm",
                                       "mxfp4_linear", "gemm16", "gemm16_grad", "gemm16_grouped",
                                       "gemm16_grouped_grad", "gemm16_weight_grad", "act16_grad")))
            _calls = module
    return _calls


def mxfp4_codes_size(rows, cols) -> int:
    """``fgemm_mxfp4_codes_size``: bytes of the codes of a rows x cols quantised matrix."""
    return int(library().fgemm_mxfp4_codes_size(rows, cols))


def mxfp4_scales_size(rows, cols) -> int:
    """``fgemm_mxfp4_scales_size``: bytes of the scales of a rows x cols quantised matrix."""
    return int(library().fgemm_mxfp4_scales_size(rows, cols))


def mxfp4_quantize(type, M, N, X, ldx, row_codes, ld_row_codes, row_scales, col_codes,
                   ld_col_codes, col_scales, stream=None, check=True) -> int:
    """``fgemm_mxfp4_quantize``: X along its rows, its columns (the quantised X^T) or both;
    None for the codes and scales of a direction that is not wanted."""
    st = (_calls or _native()).quantize(type, M, N, X, ldx, row_codes, ld_row_codes, row_scales,
                                       col_codes, ld_col_codes, col_scales, stream)
    if check:
        _check(st, "fgemm_mxfp4_quantize")
    return st


def mxfp4_quantize_grad_workspace_size(M, N) -> int:
    """``fgemm_mxfp4_quantize_grad_workspace_size``: bytes for the bias gradient's partial sums."""
    return int(library().fgemm_mxfp4_quantize_grad_workspace_size(M, N))


def mxfp4_quantize_grad(type, M, N, G, ldg, Y, ldy, row_codes, ld_row_codes, row_scales,
                        col_codes, ld_col_codes, col_scales, bias_grad, workspace,
                        workspace_bytes, stream=None, check=True) -> int:
    """``fgemm_mxfp4_quantize_grad``: G where Y > 0 (Y None: G), quantised as by
    ``mxfp4_quantize``, and its column sums (bias_grad None: not wanted)."""
    st = (_calls or _native()).quantize_grad(
        type, M, N, G, ldg, Y, ldy, row_codes, ld_row_codes, row_scales, col_codes, ld_col_codes,
        col_scales, bias_grad, workspace, workspace_bytes, stream)
    if check:
        _check(st, "fgemm_mxfp4_quantize_grad")
    return st


def mxfp4_dequantize(type, M, N, codes, ld_codes, scales, X, ldx, stream=None, check=True) -> int:
    """``fgemm_mxfp4_dequantize``: X = the values of a quantised matrix."""
    st = (_calls or _native()).dequantize(type, M, N, codes, ld_codes, scales, X, ldx, stream)
    if check:
        _check(st, "fgemm_mxfp4_dequantize")
    return st


def mxfp4_gemm(type, M, N, K, alpha, A_codes, ld_A_codes, A_scales, B_codes, ld_B_codes,
               B_scales, beta, C, ldc, bias=None, apply_relu=False, stream=None,
               check=True) -> int:
    """``fgemm_mxfp4_gemm``: C = relu?(alpha*A*B^T + beta*C + bias[col]), A and B quantised."""
    st = (_calls or _native()).gemm(type, M, N, K, alpha, A_codes, ld_A_codes, A_scales, B_codes,
                                   ld_B_codes, B_scales, beta, C, ldc, bias, apply_relu, stream)
    if check:
        _check(st, "fgemm_mxfp4_gemm")
    return st


def mxfp4_plan(type, M, N, K, num_sms) -> int:
    """``fgemm_mxfp4_plan``: 16 * tile + ranks of mxfp4_gemm's kernel for a product; host-only."""
    return library().fgemm_mxfp4_plan(type, M, N, K, num_sms)


def mxfp4_linear_workspace_size(M, N, K) -> int:
    """``fgemm_mxfp4_linear_workspace_size``: bytes of workspace mxfp4_linear needs."""
    return int(library().fgemm_mxfp4_linear_workspace_size(M, N, K))


def mxfp4_linear(type, M, N, K, X, ldx, W_codes, ld_W_codes, W_scales, bias, apply_relu, Y, ldy,
                 workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_mxfp4_linear``: Y = relu?(Q(X)*W^T + bias[col]), X quantised on the way."""
    st = (_calls or _native()).linear(type, M, N, K, X, ldx, W_codes, ld_W_codes, W_scales, bias,
                                     apply_relu, Y, ldy, workspace, workspace_bytes, stream)
    if check:
        _check(st, "fgemm_mxfp4_linear")
    return st


# ---- 16-bit layers (see "16-bit layers" in include/fgemm.h) ---------------------------

# A, B, Z, G and D are tensors of `type`, R and Y (C) of `out_type`, bias and col_sums float32, offsets
# int32 on the device; any of them may be an address.  Through the C module, like the MXFP4 calls.


def gemm16_copy_workspace_size(transa, transb, groups, M, N, K) -> int:
    """``fgemm_gemm16_copy_workspace_size``: bytes for copies of A and B whose rows are not on 16 bytes."""
    return int(library().fgemm_gemm16_copy_workspace_size(int(transa), int(transb), groups, M, N, K))


def gemm16_sums_workspace_size(groups, M, N) -> int:
    """``fgemm_gemm16_sums_workspace_size``: bytes for the partial column sums of an M x N output."""
    return int(library().fgemm_gemm16_sums_workspace_size(groups, M, N))


def gemm16(type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, bias, act, Z, ldz, beta, R, ldr, Y, ldy,
           workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_gemm16``: Z = alpha op(A) op(B) + bias (kept unless None), Y = act(Z) + beta R."""
    st = (_calls or _native()).gemm16(type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, bias, act, Z, ldz,
                                     beta, R, ldr, Y, ldy, workspace, workspace_bytes, stream)
    if check:
        _check(st, "fgemm_gemm16")
    return st


def gemm16_grad(type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, act, Z, ldz, Y, ldy, col_sums=None,
                workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_gemm16_grad``: Y = (alpha op(A) op(B)) act'(Z), and the sums of its columns."""
    st = (_calls or _native()).gemm16_grad(type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, act, Z, ldz,
                                          Y, ldy, col_sums, workspace, workspace_bytes, stream)
    if check:
        _check(st, "fgemm_gemm16_grad")
    return st


def gemm16_grouped(type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B, ldb, strideB, bias, act, Z, ldz,
                   beta, R, ldr, Y, ldy, workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_gemm16_grouped``: ``gemm16`` with B and bias of each group of rows."""
    st = (_calls or _native()).gemm16_grouped(type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B, ldb,
                                             strideB, bias, act, Z, ldz, beta, R, ldr, Y, ldy, workspace,
                                             workspace_bytes, stream)
    if check:
        _check(st, "fgemm_gemm16_grouped")
    return st


def gemm16_grouped_grad(type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B, ldb, strideB, act, Z, ldz,
                        Y, ldy, col_sums=None, workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_gemm16_grouped_grad``: ``gemm16_grad`` with B of each group of rows."""
    st = (_calls or _native()).gemm16_grouped_grad(type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B,
                                                  ldb, strideB, act, Z, ldz, Y, ldy, col_sums, workspace,
                                                  workspace_bytes, stream)
    if check:
        _check(st, "fgemm_gemm16_grouped_grad")
    return st


def gemm16_weight_grad(type, out_type, groups, M, N, K, offsets, alpha, A, lda, G, ldg, beta, C, ldc, strideC,
                       workspace=None, workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_gemm16_weight_grad``: C_e = alpha A_e^T G_e + beta C_e over each group's rows."""
    st = (_calls or _native()).gemm16_weight_grad(type, out_type, groups, M, N, K, offsets, alpha, A, lda, G, ldg, beta,
                                                 C, ldc, strideC, workspace, workspace_bytes, stream)
    if check:
        _check(st, "fgemm_gemm16_weight_grad")
    return st


def act16_grad(type, groups, M, N, offsets, act, G, ldg, Z, ldz, D, ldd, col_sums=None, workspace=None,
               workspace_bytes=0, stream=None, check=True) -> int:
    """``fgemm_act16_grad``: D = G act'(Z), and the sums of its columns for each group."""
    st = (_calls or _native()).act16_grad(type, groups, M, N, offsets, act, G, ldg, Z, ldz, D, ldd, col_sums, workspace,
                                         workspace_bytes, stream)
    if check:
        _check(st, "fgemm_act16_grad")
    return st


def gemm16_plan(out_type, grouped, groups, M, N, K, sums, num_sms) -> int:
    """``fgemm_gemm16_plan``: 16 * rows of a tile + ranks (+ 8192: pairs, + 16384: in turns); host-only."""
    return library().fgemm_gemm16_plan(out_type, grouped, groups, M, N, K, 1 if sums else 0, num_sms)
