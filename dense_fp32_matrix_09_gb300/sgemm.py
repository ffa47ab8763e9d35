"""ctypes binding of libsgemm.so, with the entry-point names of include/sgemm.h.

Argument marshalling only: every step of C = alpha*A*B + beta*C, of the int8 and
4-bit products, the norm and the expert calls runs in the CUDA library.  Matrix arguments may be raw device addresses (int) or objects
with ``data_ptr()`` (torch tensors); streams may be an int handle, a
``torch.cuda.Stream`` or ``None`` (torch's current stream).  A non-zero
status raises ``SgemmError``.  If the library has not been built the first
call raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
import typing

from . import build as _build

OK = 0
ERR_NULL = 1
ERR_INVALID_VALUE = 2
ERR_ALIAS = 3
ERR_BAD_HANDLE = 4
ERR_UNSUPPORTED_DEVICE = 5
ERR_LAUNCH = 6
ERR_CUDA = 7
ERR_DEVICE_TIMEOUT = 8
ERR_WRONG_DEVICE = 9
ERR_SCRATCH_TOO_SMALL = 10
ERR_DEVICE_CHECK = 11

VARIANT_AUTO = 0
VARIANT_TMA_128x256 = 1
VARIANT_TMA_128x128 = 2
VARIANT_TMA_64x64 = 3
VARIANT_TMA_64x64_SPLITK = 4
VARIANT_GENERIC = 5
VARIANT_SCALE = 6
VARIANT_TC_3XTF32 = 7
VARIANT_TC_3XTF32_PAIR = 8
VARIANT_TC_F16_PAIR = 9
VARIANT_GENERIC_F16 = 10
VARIANT_TMA_256x128 = 11
VARIANT_TC_I8 = 12
VARIANT_GENERIC_I8 = 13
VARIANT_FEW_I8 = 14
VARIANT_TC_F4 = 15
VARIANT_TC_F4_PAIR = 16
VARIANT_GENERIC_F4 = 17
VARIANT_COUNT = 18
MATH_FP32 = 0
MATH_3XTF32 = 1
IN_F32 = 0
IN_BF16 = 1
IN_F16 = 2
FP4_MX = 0
FP4_NV = 1
RELAYOUT_AUTO = 0
RELAYOUT_OFF = 1
RELAYOUT_ALWAYS = 2
# sgemm_sk_sums_t: how a stream-K tile's parts are added (test hook)
SK_SUMS_AUTO, SK_SUMS_LAST, SK_SUMS_DEFERRED, SK_SUMS_SHARED = 0, 1, 2, 3
GEMM_VARIANTS = (VARIANT_TMA_256x128, VARIANT_TMA_128x256, VARIANT_TMA_128x128, VARIANT_TMA_64x64,
                 VARIANT_TMA_64x64_SPLITK, VARIANT_GENERIC, VARIANT_TC_3XTF32, VARIANT_TC_3XTF32_PAIR)

#: Every exported entry point of include/sgemm.h.
EXPORTS = ("sgemm_create", "sgemm_run", "sgemm_check_args", "sgemm_destroy", "sgemm_set_variant",
           "sgemm_last_variant", "sgemm_get_device_status", "sgemm_debug_timeout_probe",
           "sgemm_debug_set_smem_override", "sgemm_status_string", "sgemm_variant_name",
           "sgemm_version", "sgemm_run_noalloc", "sgemm_set_math_mode", "sgemm_run_host",
           "sgemm_run_ex", "sgemm_check_args_ex", "sgemm_last_launches", "sgemm_run_mixed",
           "sgemm_check_args_mixed", "sgemm_debug_fma_probe", "sgemm_debug_bank_probe",
           "sgemm_set_relayout", "sgemm_last_relayout", "sgemm_relayout_capacity", "sgemm_debug_plan",
           "sgemm_debug_set_stream_k_sums", "sgemm_debug_set_cluster_split", "sgemm_debug_set_stream_k_ctas",
           "sgemm_debug_set_stream_k_gap", "sgemm_debug_leave_aborted_state", "sgemm_debug_tf32_probe",
           "sgemm_debug_set_workspace_limit", "sgemm_debug_set_int8_tile", "sgemm_run_int8", "sgemm_check_args_int8",
           "sgemm_run_int8_experts", "sgemm_check_args_int8_experts", "sgemm_quantize_rows", "sgemm_expert_sort",
           "sgemm_expert_dispatch", "sgemm_expert_dispatch_int8", "sgemm_expert_dispatch_grad",
           "sgemm_expert_combine", "sgemm_expert_combine_grad", "sgemm_quantize_fp4", "sgemm_dequantize_fp4",
           "sgemm_fp4_scale_bytes", "sgemm_run_fp4", "sgemm_check_args_fp4", "sgemm_rms_norm", "sgemm_rms_norm_int8",
           "sgemm_rms_norm_fp4", "sgemm_rms_norm_grad", "sgemm_expert_layer_int8", "sgemm_debug_set_fp4_tile")


class SgemmError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}" if where else status_string(status))


_lib = None
_calls = None          # the compiled marshalling module of the enqueue calls, when built
_calls_tried = False


def library_path() -> str:
    """The library to load: the in-tree build, or the file named by the
    SGEMM_LIBRARY environment variable (a build of the same sources with
    other flags, such as the device-checked build)."""
    return os.environ.get("SGEMM_LIBRARY") or _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it was never built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (dense_fp32_matrix_09_gb300.build.build())")
        L = ctypes.CDLL(path)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.sgemm_create.argtypes = [ctypes.POINTER(vp)]
        L.sgemm_run.argtypes = [vp, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp]
        L.sgemm_check_args.argtypes = [i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32]
        L.sgemm_destroy.argtypes = [vp]
        L.sgemm_set_variant.argtypes = [vp, i32]
        L.sgemm_last_variant.argtypes = [vp, ctypes.POINTER(i32)]
        L.sgemm_last_launches.argtypes = [vp]
        L.sgemm_set_relayout.argtypes = [vp, i32]
        L.sgemm_last_relayout.argtypes = [vp]
        L.sgemm_relayout_capacity.argtypes = [vp]
        L.sgemm_relayout_capacity.restype = ctypes.c_longlong
        L.sgemm_debug_plan.argtypes = [i32, ctypes.POINTER(i32), ctypes.c_longlong, i32, i32, i32, i32, i32, i32, i32,
                                       i32, f32, i32, ctypes.c_longlong, ctypes.c_longlong, i32, ctypes.POINTER(i32)]
        L.sgemm_debug_fma_probe.argtypes = [vp, i32, i32, vp, ctypes.POINTER(ctypes.c_longlong), vp]
        L.sgemm_debug_tf32_probe.argtypes = [vp, i32, i32, ctypes.POINTER(ctypes.c_longlong), vp]
        L.sgemm_debug_bank_probe.argtypes = [vp, i32, i32, i32, vp, vp]
        L.sgemm_run_mixed.argtypes = [vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp]
        L.sgemm_check_args_mixed.argtypes = [i32, i32, i32, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32]
        L.sgemm_get_device_status.argtypes = [vp]
        L.sgemm_debug_timeout_probe.argtypes = [vp, ctypes.c_longlong, vp]
        L.sgemm_debug_set_smem_override.argtypes = [vp, i32]
        L.sgemm_debug_set_stream_k_sums.argtypes = [vp, i32]
        L.sgemm_debug_set_cluster_split.argtypes = [vp, i32]
        L.sgemm_debug_set_int8_tile.argtypes = [vp, i32, i32]
        L.sgemm_debug_set_stream_k_ctas.argtypes = [vp, i32]
        L.sgemm_debug_set_stream_k_gap.argtypes = [vp, i32]
        L.sgemm_debug_leave_aborted_state.argtypes = [vp]
        L.sgemm_debug_set_workspace_limit.argtypes = [vp, i32]
        L.sgemm_status_string.argtypes = [i32]
        L.sgemm_status_string.restype = ctypes.c_char_p
        L.sgemm_variant_name.argtypes = [i32]
        L.sgemm_variant_name.restype = ctypes.c_char_p
        L.sgemm_version.argtypes = []
        L.sgemm_set_math_mode.argtypes = [vp, i32]
        i64 = ctypes.c_longlong
        L.sgemm_run_ex.argtypes = [vp, i32, i32, i32, i32, i32, f32, vp, i32, i64, vp, i32, i64, f32, vp, i32, i64,
                                   i32, vp]
        L.sgemm_check_args_ex.argtypes = [i32, i32, i32, i32, i32, f32, vp, i32, i64, vp, i32, i64, f32, vp, i32,
                                          i64, i32]
        L.sgemm_run_host.argtypes = [vp, i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp, vp, vp, vp]
        L.sgemm_run_noalloc.argtypes = [i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp]
        int8_args = [i32, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp, i32]
        L.sgemm_run_int8.argtypes = [vp, *int8_args, vp]
        L.sgemm_check_args_int8.argtypes = int8_args
        experts_args = [i32, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, i32, i64, vp, vp, vp, i32]
        L.sgemm_run_int8_experts.argtypes = [vp, *experts_args, vp]
        L.sgemm_check_args_int8_experts.argtypes = experts_args
        L.sgemm_quantize_rows.argtypes = [vp, i32, i32, i32, vp, i32, vp, i32, vp, vp]
        L.sgemm_expert_sort.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp]
        L.sgemm_expert_dispatch.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp]
        L.sgemm_expert_dispatch_int8.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp, vp]
        L.sgemm_expert_dispatch_grad.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp, i32, vp]
        L.sgemm_expert_combine.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp, vp, i32, vp]
        L.sgemm_expert_combine_grad.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp]
        L.sgemm_quantize_fp4.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, i32, vp, vp, vp]
        L.sgemm_dequantize_fp4.argtypes = [vp, i32, i32, i32, i32, vp, i32, vp, vp, vp, i32, vp]
        L.sgemm_fp4_scale_bytes.argtypes = [i32, i32, i32]
        L.sgemm_fp4_scale_bytes.restype = i64
        fp4_args = [i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, i32]
        L.sgemm_run_fp4.argtypes = [vp, *fp4_args, vp]
        L.sgemm_check_args_fp4.argtypes = fp4_args
        norm_in = [i32, i32, vp, i32, vp, i32, vp, f32, vp, i32]
        L.sgemm_rms_norm.argtypes = [vp, i32, *norm_in, vp, i32, vp, vp]
        L.sgemm_rms_norm_int8.argtypes = [vp, i32, *norm_in, vp, i32, vp, vp]
        L.sgemm_rms_norm_fp4.argtypes = [vp, i32, i32, *norm_in, vp, i32, vp, vp, vp]
        L.sgemm_rms_norm_grad.argtypes = [vp, i32, i32, i32, vp, i32, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp]
        L.sgemm_expert_layer_int8.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp,
                                              vp, i32, vp]
        L.sgemm_debug_set_fp4_tile.argtypes = [vp, i32, i32]
        _lib = L
    return _lib


_raw_stream = None     # (raw stream of a device, current device) of torch's bindings, once CUDA is up


def _current_stream_handle() -> int:
    """The current stream's handle.  torch.cuda.current_stream() builds a Stream
    object (2.9 us on the GB300's host, as much as a small call takes in all); the
    two calls beneath it give the handle alone (0.3 us)."""
    global _raw_stream
    if _raw_stream is not None:
        return _raw_stream[0](_raw_stream[1]())
    import torch
    handle = int(torch.cuda.current_stream().cuda_stream)   # initialises CUDA where that is still to be done
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None and raw(device()) == handle:
        _raw_stream = (raw, device)
    return handle


def calls_module():
    """The CPython module that marshals the arguments of the enqueue calls
    (built next to the library by build.py), bound to the loaded library; None
    when it was not built -- the calls then go through ctypes."""
    global _calls, _calls_tried
    if not _calls_tried:
        _calls_tried = True
        path = _build.CALLS
        if os.path.exists(path):
            import importlib.util
            lib()  # the library is loaded first; the module binds the same instance by path
            try:
                spec = importlib.util.spec_from_file_location("_sgemm_calls", path)
                mod = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(mod)
                mod.init(library_path(), _current_stream_handle)
                _calls = mod
            except (ImportError, OSError):
                _calls = None  # a module built for another interpreter or machine: ctypes serves
    return _calls


def _ptr(x) -> int | None:
    """Address of a buffer: an int, a torch tensor (data_ptr) or a numpy array."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x.__array_interface__["data"][0])


def _stream(s) -> int:
    if s is None:
        return _current_stream_handle()
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(rc: int, where: str) -> int:
    if rc != OK:
        raise SgemmError(rc, where)
    return rc


def status_string(status: int) -> str:
    return lib().sgemm_status_string(int(status)).decode()


def variant_name(variant: int) -> str:
    return lib().sgemm_variant_name(int(variant)).decode()


def sgemm_version() -> int:
    return lib().sgemm_version()


def sgemm_create() -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib().sgemm_create(ctypes.byref(h)), "sgemm_create")
    return h


def sgemm_destroy(h) -> None:
    _check(lib().sgemm_destroy(h), "sgemm_destroy")


def sgemm_run(h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*A*B + beta*C on device buffers (row-major, leading dims)."""
    calls = _calls if _calls is not None else calls_module()
    if calls is not None:
        rc = calls.run(h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)
    else:
        rc = lib().sgemm_run(h, int(M), int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B),
                             int(ldb), float(beta), _ptr(C), int(ldc), _stream(stream))
    if rc != OK:
        raise SgemmError(rc, "sgemm_run")


def sgemm_run_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*A*B + beta*C without allocating anything (no handle; fixed
    in-library scratch, at most 512 output tiles of 64 x 64).  For callers that
    cannot allocate GPU memory; see include/sgemm.h for the sharing rules."""
    _check(lib().sgemm_run_noalloc(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B),
                                   int(ldb), float(beta), _ptr(C), int(ldc), _stream(stream)),
           "sgemm_run_noalloc")


def sgemm_run_host(h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dA, dB, dC, stream=None) -> None:
    """C <- alpha*A*B + beta*C with A, B, C in host memory (page-locked for
    overlap), through the device staging buffers dA, dB, dC; copies overlap
    the per-panel GEMMs.  C is complete once `stream` has reached the call."""
    _check(lib().sgemm_run_host(h, int(M), int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B), int(ldb),
                                float(beta), _ptr(C), int(ldc), _ptr(dA), _ptr(dB), _ptr(dC), _stream(stream)),
           "sgemm_run_host")


def sgemm_run_ex(h, transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc, strideC,
                 batch=1, stream=None) -> None:
    """C_b <- alpha*op(A_b)*op(B_b) + beta*C_b, b = 0..batch-1 (see include/sgemm.h)."""
    calls = _calls if _calls is not None else calls_module()
    if calls is not None:
        rc = calls.run_ex(h, transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                          strideC, batch, stream)
    else:
        rc = lib().sgemm_run_ex(h, int(transA), int(transB), int(M), int(N), int(K), float(alpha), _ptr(A),
                                int(lda), int(strideA), _ptr(B), int(ldb), int(strideB), float(beta), _ptr(C),
                                int(ldc), int(strideC), int(batch), _stream(stream))
    if rc != OK:
        raise SgemmError(rc, "sgemm_run_ex")


def sgemm_check_args_ex(transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc, strideC,
                        batch=1) -> int:
    return lib().sgemm_check_args_ex(int(transA), int(transB), int(M), int(N), int(K), float(alpha), _ptr(A),
                                     int(lda), int(strideA), _ptr(B), int(ldb), int(strideB), float(beta), _ptr(C),
                                     int(ldc), int(strideC), int(batch))


def sgemm_check_args(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc) -> int:
    """Host-only validation; returns the status sgemm_run would return for these arguments."""
    return lib().sgemm_check_args(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B),
                                  int(ldb), float(beta), _ptr(C), int(ldc))


def sgemm_set_variant(h, variant: int) -> None:
    _check(lib().sgemm_set_variant(h, int(variant)), "sgemm_set_variant")


def sgemm_set_math_mode(h, mode: int) -> None:
    _check(lib().sgemm_set_math_mode(h, int(mode)), "sgemm_set_math_mode")


def sgemm_last_variant(h) -> tuple[int, int]:
    splits = ctypes.c_int(0)
    v = lib().sgemm_last_variant(h, ctypes.byref(splits))
    return v, splits.value


def sgemm_run_mixed(h, in_type, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C <- alpha*op(A)*op(B) + beta*C with 16-bit A, B and FP32 C (see include/sgemm.h)."""
    _check(lib().sgemm_run_mixed(h, int(in_type), int(transA), int(transB), int(M), int(N), int(K), float(alpha),
                                 _ptr(A), int(lda), _ptr(B), int(ldb), float(beta), _ptr(C), int(ldc),
                                 _stream(stream)), "sgemm_run_mixed")


def sgemm_check_args_mixed(in_type, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc) -> int:
    return lib().sgemm_check_args_mixed(int(in_type), int(transA), int(transB), int(M), int(N), int(K),
                                        float(alpha), _ptr(A), int(lda), _ptr(B), int(ldb), float(beta), _ptr(C),
                                        int(ldc))


def _integer(x, kind) -> int:
    """The value of an integer of any type (numpy's, which are buffers too, among
    them) for a parameter of the C integer type `kind`."""
    v = operator.index(x)
    if kind(v).value != v:
        raise OverflowError(f"{v} does not fit in a C {kind.__name__[2:]}")
    return v


def _enqueue(name: str, h, args, stream) -> None:
    """Call an enqueue function of the library through the marshalling module
    (every argument an int or a buffer), or through ctypes without it."""
    calls = _calls if _calls is not None else calls_module()
    if calls is not None:
        rc = calls.enqueue(name, h, args, stream)
    else:
        fn = getattr(lib(), name)
        values = [_ptr(a) if kind is ctypes.c_void_p else float(a) if kind is ctypes.c_float else _integer(a, kind)
                  for a, kind in zip(args, fn.argtypes[1:-1])]
        rc = fn(h, *values, _stream(stream))
    if rc != OK:
        raise SgemmError(rc, name)


def sgemm_run_int8(h, transB, out_type, M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, C, ldc, stream=None) -> None:
    """C = scaleA * scaleB * (A @ op(B)) + bias with int8 A and B (see include/sgemm.h)."""
    _enqueue("sgemm_run_int8", h, (transB, out_type, M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, C, ldc), stream)


def sgemm_check_args_int8(transB, out_type, M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, C, ldc) -> int:
    return lib().sgemm_check_args_int8(int(transB), int(out_type), int(M), int(N), int(K), _ptr(A), int(lda),
                                       _ptr(scaleA), _ptr(B), int(ldb), _ptr(scaleB), _ptr(bias), _ptr(C), int(ldc))


def sgemm_run_int8_experts(h, transB, out_type, experts, rows, N, K, offsets, A, lda, scaleA, B, ldb, strideB,
                           scaleB, bias, C, ldc, stream=None) -> None:
    """The int8 product over rows sorted by expert, each expert with its own B
    (offsets: experts + 1 ints on the device; see include/sgemm.h)."""
    _enqueue("sgemm_run_int8_experts", h, (transB, out_type, experts, rows, N, K, offsets, A, lda, scaleA, B, ldb,
                                           strideB, scaleB, bias, C, ldc), stream)


def sgemm_check_args_int8_experts(transB, out_type, experts, rows, N, K, offsets, A, lda, scaleA, B, ldb, strideB,
                                  scaleB, bias, C, ldc) -> int:
    return lib().sgemm_check_args_int8_experts(
        int(transB), int(out_type), int(experts), int(rows), int(N), int(K), _ptr(offsets), _ptr(A), int(lda),
        _ptr(scaleA), _ptr(B), int(ldb), int(strideB), _ptr(scaleB), _ptr(bias), _ptr(C), int(ldc))


def sgemm_quantize_rows(h, in_type, M, K, X, ldx, Q, ldq, scale, stream=None) -> None:
    """Q (int8), scale (FP32) = the rows of X, each divided by its scale and rounded."""
    _enqueue("sgemm_quantize_rows", h, (in_type, M, K, X, ldx, Q, ldq, scale), stream)


def sgemm_expert_sort(h, tokens, choices, experts, ids, offsets, rows, source, stream=None) -> None:
    """The (token, choice) slots in a stable order by expert."""
    _enqueue("sgemm_expert_sort", h, (tokens, choices, experts, ids, offsets, rows, source), stream)


def sgemm_expert_dispatch(h, in_type, tokens, choices, width, X, ldx, rows, Y, ldy, stream=None) -> None:
    """Y[rows[t, j]] = X[t]."""
    _enqueue("sgemm_expert_dispatch", h, (in_type, tokens, choices, width, X, ldx, rows, Y, ldy), stream)


def sgemm_expert_dispatch_int8(h, in_type, tokens, choices, width, X, ldx, rows, Q, ldq, scale, stream=None) -> None:
    """Q[rows[t, j]], scale[rows[t, j]] = row t of X, quantized."""
    _enqueue("sgemm_expert_dispatch_int8", h, (in_type, tokens, choices, width, X, ldx, rows, Q, ldq, scale), stream)


def sgemm_expert_dispatch_grad(h, in_type, tokens, choices, width, dY, lddy, rows, dX, lddx, stream=None) -> None:
    """dX[t] = sum_j dY[rows[t, j]]."""
    _enqueue("sgemm_expert_dispatch_grad", h, (in_type, tokens, choices, width, dY, lddy, rows, dX, lddx), stream)


def sgemm_expert_combine(h, in_type, tokens, choices, width, Y, ldy, rows, weights, out, ldo, stream=None) -> None:
    """out[t] = sum_j weights[t, j] * Y[rows[t, j]]."""
    _enqueue("sgemm_expert_combine", h, (in_type, tokens, choices, width, Y, ldy, rows, weights, out, ldo), stream)


def sgemm_expert_combine_grad(h, in_type, tokens, choices, width, dout, lddo, Y, ldy, rows, weights, dY, lddy,
                              dweights, stream=None) -> None:
    """dY[rows[t, j]] = weights[t, j] * dout[t]; dweights[t, j] = <dout[t], Y[rows[t, j]]>."""
    _enqueue("sgemm_expert_combine_grad", h, (in_type, tokens, choices, width, dout, lddo, Y, ldy, rows, weights,
                                              dY, lddy, dweights), stream)


def sgemm_fp4_scale_bytes(fmt, rows, K) -> int:
    """Bytes of the scales of `rows` rows of K elements in 4 bits (-1: unknown format, bad size)."""
    return lib().sgemm_fp4_scale_bytes(int(fmt), int(rows), int(K))


def sgemm_quantize_fp4(h, in_type, fmt, M, K, X, ldx, Q, ldq, S, row, stream=None) -> None:
    """Q, S, row = the rows of X in 4-bit floating point with a scale a block (see include/sgemm.h)."""
    _enqueue("sgemm_quantize_fp4", h, (in_type, fmt, M, K, X, ldx, Q, ldq, S, row), stream)


def sgemm_dequantize_fp4(h, out_type, fmt, M, K, Q, ldq, S, row, Y, ldy, stream=None) -> None:
    """Y = what the 4-bit rows stand for."""
    _enqueue("sgemm_dequantize_fp4", h, (out_type, fmt, M, K, Q, ldq, S, row, Y, ldy), stream)


def sgemm_run_fp4(h, fmt, out_type, M, N, K, A, lda, SA, rowA, B, ldb, SB, rowB, bias, C, ldc, stream=None) -> None:
    """C = A @ B.T + bias for A and B in 4-bit floating point (see include/sgemm.h)."""
    _enqueue("sgemm_run_fp4", h, (fmt, out_type, M, N, K, A, lda, SA, rowA, B, ldb, SB, rowB, bias, C, ldc), stream)


def sgemm_check_args_fp4(fmt, out_type, M, N, K, A, lda, SA, rowA, B, ldb, SB, rowB, bias, C, ldc) -> int:
    return lib().sgemm_check_args_fp4(int(fmt), int(out_type), int(M), int(N), int(K), _ptr(A), int(lda), _ptr(SA),
                                      _ptr(rowA), _ptr(B), int(ldb), _ptr(SB), _ptr(rowB), _ptr(bias), _ptr(C), int(ldc))


def sgemm_rms_norm(h, in_type, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Y, ldy, rstd, stream=None) -> None:
    """H = X + R; Y = H * weight / rms(H), rstd = 1 / rms (see include/sgemm.h)."""
    _enqueue("sgemm_rms_norm", h, (in_type, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Y, ldy, rstd), stream)


def sgemm_rms_norm_int8(h, in_type, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, scale, stream=None) -> None:
    """The same with the result in 8 bits and a scale a row."""
    _enqueue("sgemm_rms_norm_int8", h, (in_type, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, scale), stream)


def sgemm_rms_norm_fp4(h, in_type, fmt, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, S, row, stream=None) -> None:
    """The same with the result in 4 bits, a scale a block and one a row."""
    _enqueue("sgemm_rms_norm_fp4", h, (in_type, fmt, M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, S, row), stream)


def sgemm_rms_norm_grad(h, in_type, M, K, dY, lddy, dH, lddh, H, ldh, weight, rstd, dX, lddx, dweight, stream=None) -> None:
    """dX and dweight of sgemm_rms_norm."""
    _enqueue("sgemm_rms_norm_grad", h, (in_type, M, K, dY, lddy, dH, lddh, H, ldh, weight, rstd, dX, lddx, dweight),
             stream)


def sgemm_expert_layer_int8(h, in_type, gated, tokens, choices, experts, width, hidden, X, ldx, ids, weights, up,
                            up_scale, down, down_scale, out, ldo, stream=None) -> None:
    """out[t] = sum_j weights[t, j] * down_e(act(up_e(X[t]))) for a few tokens."""
    _enqueue("sgemm_expert_layer_int8", h, (in_type, gated, tokens, choices, experts, width, hidden, X, ldx, ids,
                                            weights, up, up_scale, down, down_scale, out, ldo), stream)


def sgemm_debug_fma_probe(h, sink, ctas=0, iters=4096, stream=None) -> int:
    """Enqueue the FP32 FMA-rate probe (sink: ctas*256 floats on the device);
    returns the FLOP it performs."""
    flops = ctypes.c_longlong(0)
    _check(lib().sgemm_debug_fma_probe(h, int(ctas), int(iters), _ptr(sink), ctypes.byref(flops), _stream(stream)),
           "sgemm_debug_fma_probe")
    return flops.value


def sgemm_debug_tf32_probe(h, clusters=0, iters=4096, stream=None) -> int:
    """Enqueue the TF32 tensor-pipe rate probe; returns the TF32 FLOP it performs."""
    flops = ctypes.c_longlong(0)
    _check(lib().sgemm_debug_tf32_probe(h, int(clusters), int(iters), ctypes.byref(flops), _stream(stream)),
           "sgemm_debug_tf32_probe")
    return flops.value


def sgemm_debug_bank_probe(h, padded, sink, ctas=0, iters=64, stream=None) -> None:
    """Enqueue the shared-memory bank probe (sink: ctas*32 floats on the device)."""
    _check(lib().sgemm_debug_bank_probe(h, int(padded), int(ctas), int(iters), _ptr(sink), _stream(stream)),
           "sgemm_debug_bank_probe")


def sgemm_last_launches(h) -> int:
    return lib().sgemm_last_launches(h)


def sgemm_set_relayout(h, mode: int) -> None:
    _check(lib().sgemm_set_relayout(h, int(mode)), "sgemm_set_relayout")


def sgemm_last_relayout(h) -> int:
    """Operands the last call copied transposed first: bit 0 A, bit 1 B."""
    return lib().sgemm_last_relayout(h)


def sgemm_relayout_capacity(h) -> int:
    return lib().sgemm_relayout_capacity(h)


PLAN_FIELDS = ("kind", "variant", "copies", "op", "dp_tiles", "sk_ctas", "tiles", "launches", "splits",
               "fixup", "ksplit", "tc_bk", "sk_gap")
# "fixup": how the stream-K tiles' parts are added (0 last CTA or no stream-K, 1 second kernel, 2 shared)
FIXUP_LAST, FIXUP_DEFERRED, FIXUP_SHARED = 0, 1, 2
PLAN_NOTHING, PLAN_SCALE, PLAN_TENSOR_CORE, PLAN_GENERIC, PLAN_TMA = 0, 1, 2, 3, 4


def sgemm_debug_plan(num_sms, ctas_per_sm, transA, transB, M, N, K, *, alpha=1.0, batch=1, strideA=0,
                     strideB=0, tma_ok=True, relayout_floats=2 * 8192 * 8192, relayout_mode=RELAYOUT_AUTO,
                     math_mode=MATH_FP32, pinned=VARIANT_AUTO) -> dict:
    """The plan sgemm_run_ex would follow, computed on the host (no GPU):
    a dict with the fields of PLAN_FIELDS (see include/sgemm.h).  ``tma_ok``:
    True (both operands TMA-readable as stored), False (neither), or the
    bitmask of those that are (bit 0 A, bit 1 B)."""
    aligned = 3 if tma_ok is True else 0 if tma_ok is False else int(tma_ok)
    occ = (ctypes.c_int * VARIANT_COUNT)(*ctas_per_sm)
    out = (ctypes.c_int * len(PLAN_FIELDS))()
    _check(lib().sgemm_debug_plan(int(num_sms), occ, int(relayout_floats), int(relayout_mode), int(math_mode),
                                  int(pinned), int(transA), int(transB), int(M), int(N), int(K), float(alpha),
                                  int(batch), int(strideA), int(strideB), aligned, out),
           "sgemm_debug_plan")
    return dict(zip(PLAN_FIELDS, list(out)))


def sgemm_get_device_status(h) -> int:
    return lib().sgemm_get_device_status(h)


def sgemm_debug_timeout_probe(h, limit_ns: int, stream=None) -> None:
    _check(lib().sgemm_debug_timeout_probe(h, int(limit_ns), _stream(stream)), "sgemm_debug_timeout_probe")


def sgemm_debug_set_smem_override(h, nbytes: int) -> None:
    _check(lib().sgemm_debug_set_smem_override(h, int(nbytes)), "sgemm_debug_set_smem_override")


def sgemm_debug_set_workspace_limit(h, tiles: int) -> None:
    _check(lib().sgemm_debug_set_workspace_limit(h, int(tiles)), "sgemm_debug_set_workspace_limit")


def sgemm_debug_leave_aborted_state(h) -> None:
    _check(lib().sgemm_debug_leave_aborted_state(h), "sgemm_debug_leave_aborted_state")


def sgemm_debug_set_stream_k_ctas(h, ctas: int) -> None:
    """Test hook: stream-K CTAs of later calls' stream-K plans (0: the library's choice)."""
    _check(lib().sgemm_debug_set_stream_k_ctas(h, int(ctas)), "sgemm_debug_set_stream_k_ctas")


def sgemm_debug_set_stream_k_gap(h, gap: int) -> None:
    """Test hook: boundary charge of later calls' stream-K splits, in
    sixteenths of a K step (-1: the library's choice; 0: the even split)."""
    _check(lib().sgemm_debug_set_stream_k_gap(h, int(gap)), "sgemm_debug_set_stream_k_gap")


def sgemm_debug_set_cluster_split(h, ksplit: int) -> None:
    """0: automatic; 1: no cluster split-K; 2..8: that many CTAs per tile."""
    _check(lib().sgemm_debug_set_cluster_split(h, int(ksplit)), "sgemm_debug_set_cluster_split")


def sgemm_debug_set_int8_tile(h, tokens: int, ksplit: int) -> None:
    """Token tile and K split of later int8 products on the tensor cores (test hook; 0, 0: the library's choice)."""
    _check(lib().sgemm_debug_set_int8_tile(h, int(tokens), int(ksplit)), "sgemm_debug_set_int8_tile")


def sgemm_debug_set_fp4_tile(h, tokens: int, ksplit: int) -> None:
    """Token tile and K split of later 4-bit products on the tensor cores (test hook; 0, 0: the library's choice)."""
    _check(lib().sgemm_debug_set_fp4_tile(h, int(tokens), int(ksplit)), "sgemm_debug_set_fp4_tile")


def sgemm_debug_set_stream_k_sums(h, mode: int) -> None:
    """mode: one of SK_SUMS_AUTO, SK_SUMS_LAST, SK_SUMS_DEFERRED, SK_SUMS_SHARED."""
    _check(lib().sgemm_debug_set_stream_k_sums(h, int(mode)), "sgemm_debug_set_stream_k_sums")


def _element_type(t) -> int:
    """The library's value of a tensor's element type (FP32, BF16, FP16)."""
    import torch
    kinds = {torch.float32: IN_F32, torch.bfloat16: IN_BF16, torch.float16: IN_F16}
    if t.dtype not in kinds:
        raise ValueError(f"FP32, BF16 or FP16 is wanted, got {t.dtype}")
    return kinds[t.dtype]


def _ld(t) -> int:
    """Leading dimension of a 2-D tensor (one row: any value that its columns fit)."""
    return max(t.stride(0), t.shape[1], 1)


def _current_device() -> int:
    if _raw_stream is not None:         # (the call beneath torch.cuda.current_device())
        return _raw_stream[1]()
    import torch
    return torch.cuda.current_device()


def _on_device(**tensors) -> None:
    """Every tensor (None: not given) is on the current CUDA device, whose addresses
    the kernels can use."""
    current = _current_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != current:   # (-1 on the host)
            raise ValueError(f"{name} must be on the current device (cuda:{current}), got {t.device}" if t.is_cuda else
                             f"{name} must be on the GPU, got {t.device}")


def _rows_of(name, t, dtype=None) -> None:
    # (of one column the stride says nothing: a contiguous tensor may have any there)
    if t.dim() != 2 or (t.numel() and t.shape[1] > 1 and t.stride(1) != 1) or \
            (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name} must be 2-D with unit column stride and rows that do not overlap")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _vector(name, t, n, dtype=None) -> None:
    import torch
    want = dtype or torch.float32
    if tuple(t.shape) != (n,) or t.dtype != want or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {want} vector of {n}, got {t.dtype} {tuple(t.shape)}")


def _weights(t, tokens, choices) -> None:
    import torch
    if tuple(t.shape) != (tokens, choices) or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"weights must be a contiguous {tokens} x {choices} FP32 tensor")


def _slots(rows, tokens=None) -> tuple[int, int]:
    import torch
    if rows.dim() != 2 or rows.dtype != torch.int32 or not rows.is_contiguous() or \
            (tokens is not None and rows.shape[0] != tokens):
        raise ValueError("rows must be a contiguous tokens x choices int32 tensor")
    return rows.shape[0], rows.shape[1]


_HERE = contextlib.nullcontext()


def _on(stream, *tensors):
    """The context in which a tensor method makes its results and enqueues its
    kernels: on `stream` everything, so that the results' memory and what fills it
    are in order with the kernels.  The memory of `tensors` (what the method reads or
    is given to write) is kept from reuse until `stream` is done with it."""
    if stream is None:
        return _HERE
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _result(out, M, N, out_dtype, device):
    import torch
    if out is None:
        return torch.empty(M, N, dtype=out_dtype or torch.bfloat16, device=device)
    _rows_of("out", out, out_dtype)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be {M} x {N}, got {tuple(out.shape)}")
    return out


class Fp4Rows(typing.NamedTuple):
    """Rows in 4-bit floating point: what the tensor methods hand round (see include/sgemm.h)."""
    Q: object        # rows x bytes, uint8: two elements a byte
    S: object        # the blocks' scales in tiles of 128 rows x 4 blocks, uint8
    row: object      # one FP32 a row, or None (MX only)
    K: int           # elements a row
    format: int      # FP4_MX or FP4_NV


def fp4_blocks(fmt, K) -> int:
    """Blocks of a row of K elements."""
    if fmt not in (FP4_MX, FP4_NV):
        raise ValueError(f"unknown 4-bit format {fmt}")
    return -(-K // (32 if fmt == FP4_MX else 16))


def fp4_tile_scales(scales, fmt, K):
    """Scale bytes of rows x blocks (uint8, as other libraries keep them) in the tiles that the 4-bit
    calls read, zeros behind the last row and block."""
    import torch
    rows, blocks = scales.shape
    if scales.dtype != torch.uint8 or blocks != fp4_blocks(fmt, K):
        raise ValueError(f"scales must be uint8, rows x {fp4_blocks(fmt, K)}, got {scales.dtype} {tuple(scales.shape)}")
    full = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=scales.device)
    full[:rows, :blocks] = scales
    return full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _fp4(name, a) -> None:
    """The parts of rows in 4 bits fit together."""
    import torch
    if a.format not in (FP4_MX, FP4_NV):
        raise ValueError(f"{name}: unknown 4-bit format {a.format}")
    _rows_of(f"{name}.Q", a.Q, torch.uint8)
    rows, need = a.Q.shape[0], sgemm_fp4_scale_bytes(a.format, a.Q.shape[0], a.K)
    if a.K < 0 or a.Q.shape[1] < (a.K + 1) // 2:
        raise ValueError(f"{name}: rows of {a.Q.shape[1]} bytes do not hold {a.K} elements")
    if a.S.dtype != torch.uint8 or a.S.dim() != 1 or not a.S.is_contiguous() or a.S.numel() < need:
        raise ValueError(f"{name}.S must be a contiguous uint8 vector of at least {need}")
    if a.row is not None:
        _vector(f"{name}.row", a.row, rows)
    elif a.format == FP4_NV:
        raise ValueError(f"{name}.row is wanted with FP4_NV")


class Sgemm:
    """A handle as a context manager: ``with Sgemm() as g: g.run(...)``.

    The methods on torch tensors enqueue on `stream` (None: torch's current one).
    Those that return new tensors make them there, as torch does under
    ``torch.cuda.stream(stream)``: the inputs have to be ready on that stream, and
    another stream that uses the results has to wait for it.
    """

    def __init__(self, variant: int = VARIANT_AUTO):
        self.h = sgemm_create()
        if variant != VARIANT_AUTO:
            sgemm_set_variant(self.h, variant)

    def run(self, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
        sgemm_run(self.h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)

    def matmul(self, A, B, C, alpha=1.0, beta=0.0, stream=None):
        """C <- alpha*A@B + beta*C for 2-D row-major torch tensors (unit column stride)."""
        M, K = A.shape
        K2, N = B.shape
        if K2 != K or tuple(C.shape) != (M, N):
            raise ValueError(f"shape mismatch: {tuple(A.shape)} @ {tuple(B.shape)} -> {tuple(C.shape)}")
        for t in (A, B, C):
            if t.dim() != 2 or (t.numel() and t.stride(1) != 1):
                raise ValueError("operands must be 2-D with unit column stride")
        sgemm_run(self.h, M, N, K, alpha, A, max(A.stride(0), 1), B, max(B.stride(0), 1), beta, C,
                  max(C.stride(0), 1), stream)
        return C

    # -- 8-bit products and expert routing on torch tensors: devices, shapes and
    #    types are checked here, results are new tensors on the inputs' device ------
    def quantize(self, X, stream=None):
        """(Q, scale): the rows of X (2-D, FP32/BF16/FP16) in int8 and their FP32 scales."""
        import torch
        _on_device(X=X)
        kind = _element_type(X)
        _rows_of("X", X)
        M, K = X.shape
        with _on(stream, X):
            Q = torch.empty(M, K, dtype=torch.int8, device=X.device)
            scale = torch.empty(M, dtype=torch.float32, device=X.device)
            sgemm_quantize_rows(self.h, kind, M, K, X, _ld(X), Q, max(K, 1), scale)
        return Q, scale

    def matmul_int8(self, A, scaleA, B, scaleB, bias=None, out_dtype=None, out=None, stream=None):
        """scaleA[:, None] * scaleB * (A @ B.T) + bias for int8 A (M x K) and B (N x K);
        `out_dtype` (BF16 unless given) or `out` says of which type."""
        import torch
        _on_device(A=A, scaleA=scaleA, B=B, scaleB=scaleB, bias=bias, out=out)
        _rows_of("A", A, torch.int8)
        _rows_of("B", B, torch.int8)
        (M, K), (N, K2) = A.shape, B.shape
        if K2 != K:
            raise ValueError(f"shape mismatch: {tuple(A.shape)} @ {tuple(B.shape)}.T")
        _vector("scaleA", scaleA, M)
        _vector("scaleB", scaleB, N)
        if bias is not None:
            _vector("bias", bias, N)
        with _on(stream, A, scaleA, B, scaleB, bias, out):
            out = _result(out, M, N, out_dtype, A.device)
            sgemm_run_int8(self.h, 1, _element_type(out), M, N, K, A, _ld(A), scaleA, B, _ld(B), scaleB, bias, out,
                           _ld(out))
        return out

    def matmul_int8_experts(self, offsets, A, scaleA, B, scaleB, bias=None, out_dtype=None, out=None, stream=None):
        """As matmul_int8 for rows sorted by expert: rows offsets[e] .. offsets[e+1]-1
        of A with B[e] (experts x N x K, contiguous); scaleB, bias: experts x N.  Rows of
        no expert are left as they are in `out` (zeros without it)."""
        import torch
        _on_device(offsets=offsets, A=A, scaleA=scaleA, B=B, scaleB=scaleB, bias=bias, out=out)
        _rows_of("A", A, torch.int8)
        if B.dim() != 3 or B.dtype != torch.int8 or not B.is_contiguous() or B.shape[2] != A.shape[1]:
            raise ValueError(f"B must be a contiguous experts x N x {A.shape[1]} int8 tensor, got {tuple(B.shape)}")
        (E, N, K), R = B.shape, A.shape[0]
        _vector("offsets", offsets, E + 1, torch.int32)
        _vector("scaleA", scaleA, R)
        for name, t in (("scaleB", scaleB), ("bias", bias)):
            if t is not None and (tuple(t.shape) != (E, N) or t.dtype != torch.float32 or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {E} x {N} FP32 tensor")
        with _on(stream, offsets, A, scaleA, B, scaleB, bias, out):
            if out is None:
                out = torch.zeros(R, N, dtype=out_dtype or torch.bfloat16, device=A.device)
            out = _result(out, R, N, out_dtype, A.device)
            sgemm_run_int8_experts(self.h, 1, _element_type(out), E, R, N, K, offsets, A, _ld(A), scaleA, B, max(K, 1),
                                   N * K, scaleB, bias, out, _ld(out))
        return out

    def expert_sort(self, ids, experts, stream=None):
        """(offsets, rows, source) of ids (tokens x choices, int32)."""
        import torch
        _on_device(ids=ids)
        if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous tokens x choices int32 tensor")
        tokens, choices = ids.shape
        with _on(stream, ids):
            offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
            rows = torch.empty(tokens, choices, dtype=torch.int32, device=ids.device)
            source = torch.empty(tokens * choices, dtype=torch.int32, device=ids.device)
            sgemm_expert_sort(self.h, tokens, choices, experts, ids, offsets, rows, source)
        return offsets, rows, source

    def expert_dispatch(self, X, rows, stream=None):
        """The tokens' rows in the experts' order (tokens * choices rows; those of no slot are zero)."""
        import torch
        _on_device(X=X, rows=rows)
        _rows_of("X", X)
        tokens, choices = _slots(rows, X.shape[0])
        with _on(stream, X, rows):
            Y = torch.zeros(tokens * choices, X.shape[1], dtype=X.dtype, device=X.device)
            sgemm_expert_dispatch(self.h, _element_type(X), tokens, choices, X.shape[1], X, _ld(X), rows, Y, _ld(Y))
        return Y

    def expert_dispatch_int8(self, X, rows, stream=None):
        """(Q, scale): expert_dispatch and quantize in one pass."""
        import torch
        _on_device(X=X, rows=rows)
        _rows_of("X", X)
        tokens, choices = _slots(rows, X.shape[0])
        with _on(stream, X, rows):
            Q = torch.zeros(tokens * choices, X.shape[1], dtype=torch.int8, device=X.device)
            scale = torch.zeros(tokens * choices, dtype=torch.float32, device=X.device)
            sgemm_expert_dispatch_int8(self.h, _element_type(X), tokens, choices, X.shape[1], X, _ld(X), rows, Q,
                                       _ld(Q), scale)
        return Q, scale

    def expert_dispatch_grad(self, dY, rows, stream=None):
        """dX from the gradient of expert_dispatch's result."""
        import torch
        _on_device(dY=dY, rows=rows)
        tokens, choices = _slots(rows)
        _rows_of("dY", dY)
        if dY.shape[0] != tokens * choices:
            raise ValueError(f"dY must have {tokens * choices} rows, got {dY.shape[0]}")
        with _on(stream, dY, rows):
            dX = torch.empty(tokens, dY.shape[1], dtype=dY.dtype, device=dY.device)
            sgemm_expert_dispatch_grad(self.h, _element_type(dY), tokens, choices, dY.shape[1], dY, _ld(dY), rows, dX,
                                       _ld(dX))
        return dX

    def expert_combine(self, Y, rows, weights, stream=None):
        """sum_j weights[t, j] * Y[rows[t, j]]."""
        import torch
        _on_device(Y=Y, rows=rows, weights=weights)
        tokens, choices = _slots(rows)
        _rows_of("Y", Y)
        _weights(weights, tokens, choices)
        if Y.shape[0] != tokens * choices:
            raise ValueError(f"Y must have {tokens * choices} rows, got {Y.shape[0]}")
        with _on(stream, Y, rows, weights):
            out = torch.empty(tokens, Y.shape[1], dtype=Y.dtype, device=Y.device)
            sgemm_expert_combine(self.h, _element_type(Y), tokens, choices, Y.shape[1], Y, _ld(Y), rows, weights, out,
                                 _ld(out))
        return out

    def expert_combine_grad(self, dout, Y, rows, weights, stream=None):
        """(dY, dweights) of expert_combine; rows of no slot have a zero gradient."""
        import torch
        _on_device(dout=dout, Y=Y, rows=rows, weights=weights)
        tokens, choices = _slots(rows, dout.shape[0])
        _rows_of("dout", dout, Y.dtype)
        _rows_of("Y", Y)
        _weights(weights, tokens, choices)
        if tuple(Y.shape) != (tokens * choices, dout.shape[1]):
            raise ValueError(f"Y must be {tokens * choices} x {dout.shape[1]}, got {tuple(Y.shape)}")
        with _on(stream, dout, Y, rows, weights):
            dY = torch.zeros_like(Y, memory_format=torch.contiguous_format)
            dweights = torch.empty(tokens, choices, dtype=torch.float32, device=Y.device)
            sgemm_expert_combine_grad(self.h, _element_type(Y), tokens, choices, Y.shape[1], dout, _ld(dout), Y, _ld(Y),
                                      rows, weights, dY, _ld(dY), dweights)
        return dY, dweights

    # -- 4-bit floating point, the RMS norm and the whole expert layer --------------------
    def quantize_fp4(self, X, format=FP4_MX, stream=None):
        """The rows of X (2-D, FP32/BF16/FP16) in 4 bits, as Fp4Rows (row scales with FP4_NV)."""
        _on_device(X=X)
        kind = _element_type(X)
        _rows_of("X", X)
        with _on(stream, X):
            out = self._fp4_out(X, format, format == FP4_NV)
            sgemm_quantize_fp4(self.h, kind, format, X.shape[0], X.shape[1], X, _ld(X), out.Q, _ld(out.Q), out.S, out.row)
        return out

    @staticmethod
    def _fp4_out(X, format, with_row):
        import torch
        (M, K), new = X.shape, dict(device=X.device)
        n = sgemm_fp4_scale_bytes(format, M, K)
        if n < 0:
            raise ValueError(f"unknown 4-bit format {format}")
        # rows on 16-byte boundaries; scales of rows behind the last, which the kernels leave alone, are
        # zeros, so that the whole buffer may be stored or compared
        return Fp4Rows(torch.empty(M, max(-(-K // 32) * 16, 1), dtype=torch.uint8, **new), torch.zeros(n, dtype=torch.uint8, **new),
                       # (rows of no elements are not touched: their products are 0)
                       (torch.empty if K else torch.zeros)(M, dtype=torch.float32, **new) if with_row else None, K, format)

    def dequantize_fp4(self, A, out_dtype=None, out=None, stream=None):
        """What 4-bit rows stand for (BF16 unless `out_dtype` or `out` says otherwise)."""
        _on_device(Q=A.Q, S=A.S, row=A.row, out=out)
        _fp4("A", A)
        M = A.Q.shape[0]
        with _on(stream, A.Q, A.S, A.row, out):
            out = _result(out, M, A.K, out_dtype, A.Q.device)
            sgemm_dequantize_fp4(self.h, _element_type(out), A.format, M, A.K, A.Q, _ld(A.Q), A.S, A.row, out, _ld(out))
        return out

    def matmul_fp4(self, A, B, bias=None, out_dtype=None, out=None, stream=None):
        """A @ B.T + bias for A (M rows) and B (N rows) in the same 4-bit format; `out_dtype` (BF16
        unless given) or `out` says of which type."""
        _on_device(**{"A.Q": A.Q, "A.S": A.S, "A.row": A.row, "B.Q": B.Q, "B.S": B.S, "B.row": B.row, "bias": bias, "out": out})
        _fp4("A", A)
        _fp4("B", B)
        if A.K != B.K or A.format != B.format:
            raise ValueError(f"A and B differ: {A.K} and {B.K} elements a row, formats {A.format} and {B.format}")
        M, N = A.Q.shape[0], B.Q.shape[0]
        if bias is not None:
            _vector("bias", bias, N)
        with _on(stream, A.Q, A.S, A.row, B.Q, B.S, B.row, bias, out):
            out = _result(out, M, N, out_dtype, A.Q.device)
            sgemm_run_fp4(self.h, A.format, _element_type(out), M, N, A.K, A.Q, _ld(A.Q), A.S, A.row, B.Q, _ld(B.Q), B.S,
                          B.row, bias, out, _ld(out))
        return out

    @staticmethod
    def _norm_rows(X, weight, residual):
        _on_device(X=X, weight=weight, residual=residual)
        _element_type(X)
        _rows_of("X", X)
        _vector("weight", weight, X.shape[1], X.dtype)
        if residual is not None:
            _rows_of("residual", residual, X.dtype)
            if residual.shape != X.shape:
                raise ValueError(f"residual must be {tuple(X.shape)}, got {tuple(residual.shape)}")

    @staticmethod
    def _norm_args(X, weight, residual, eps, H):
        return (X, _ld(X), residual, _ld(residual) if residual is not None else 0, weight, eps, H,
                _ld(H) if H is not None else 0)

    def rms_norm(self, X, weight, residual=None, eps=1e-5, stream=None):
        """(Y, H, rstd): H = X + residual (X itself without one), Y = H * weight / rms(H), rstd = 1 / rms."""
        import torch
        self._norm_rows(X, weight, residual)
        M, K = X.shape
        with _on(stream, X, weight, residual):
            Y = torch.empty(M, K, dtype=X.dtype, device=X.device)
            H = torch.empty_like(Y) if residual is not None else None
            # (rows of no elements are not touched)
            rstd = torch.empty(M, dtype=torch.float32, device=X.device) if K else torch.zeros(M, device=X.device)
            sgemm_rms_norm(self.h, _element_type(X), M, K, *self._norm_args(X, weight, residual, eps, H), Y, _ld(Y), rstd)
        return Y, X if H is None else H, rstd

    def rms_norm_int8(self, X, weight, residual=None, eps=1e-5, stream=None):
        """(Q, scale, H): the normed rows in 8 bits with a scale a row, and H."""
        import torch
        self._norm_rows(X, weight, residual)
        M, K = X.shape
        with _on(stream, X, weight, residual):
            Q = torch.empty(M, K, dtype=torch.int8, device=X.device)
            scale = torch.zeros(M, dtype=torch.float32, device=X.device)
            H = torch.empty(M, K, dtype=X.dtype, device=X.device) if residual is not None else None
            sgemm_rms_norm_int8(self.h, _element_type(X), M, K, *self._norm_args(X, weight, residual, eps, H), Q, _ld(Q), scale)
        return Q, scale, X if H is None else H

    def rms_norm_fp4(self, X, weight, residual=None, eps=1e-5, format=FP4_MX, stream=None):
        """(rows, H): the normed rows in 4 bits (Fp4Rows, with row scales in either format), and H."""
        import torch
        self._norm_rows(X, weight, residual)
        M, K = X.shape
        with _on(stream, X, weight, residual):
            out = self._fp4_out(X, format, True)
            H = torch.empty(M, K, dtype=X.dtype, device=X.device) if residual is not None else None
            sgemm_rms_norm_fp4(self.h, _element_type(X), format, M, K, *self._norm_args(X, weight, residual, eps, H), out.Q,
                               _ld(out.Q), out.S, out.row)
        return out, X if H is None else H

    def rms_norm_grad(self, dY, H, weight, rstd, dH=None, stream=None):
        """(dX, dweight) of rms_norm from the gradients of its Y and, if it has one, of its H; dX is the
        gradient of X and of the residual, dweight FP32."""
        import torch
        _on_device(dY=dY, H=H, weight=weight, rstd=rstd, dH=dH)
        kind = _element_type(H)
        _rows_of("H", H)
        for name, t in (("dY", dY), ("dH", dH)):
            if t is not None:
                _rows_of(name, t, H.dtype)
                if t.shape != H.shape:
                    raise ValueError(f"{name} must be {tuple(H.shape)}, got {tuple(t.shape)}")
        M, K = H.shape
        _vector("weight", weight, K, H.dtype)
        _vector("rstd", rstd, M)
        with _on(stream, dY, H, weight, rstd, dH):
            dX = torch.empty(M, K, dtype=H.dtype, device=H.device)
            dweight = torch.empty(K, dtype=torch.float32, device=H.device)
            sgemm_rms_norm_grad(self.h, kind, M, K, dY, _ld(dY), dH, _ld(dH) if dH is not None else 0, H, _ld(H), weight,
                                rstd, dX, _ld(dX), dweight)
        return dX, dweight

    def expert_layer_int8(self, X, ids, weights, up, up_scale, down, down_scale, gated=False, stream=None):
        """sum_j weights[t, j] * down_e(act(up_e(X[t]))), e = ids[t, j], for up to 64 tokens: up (experts x
        hidden x width, with `gated` 2 * hidden: silu of the first half times the second) and down
        (experts x width x hidden) in int8 with scales a channel."""
        import torch
        _on_device(X=X, ids=ids, weights=weights, up=up, up_scale=up_scale, down=down, down_scale=down_scale)
        kind = _element_type(X)
        _rows_of("X", X)
        T, W = X.shape
        if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous() or ids.shape[0] != T:
            raise ValueError("ids must be a contiguous tokens x choices int32 tensor")
        _weights(weights, T, ids.shape[1])
        if down.dim() != 3 or down.shape[1] != W:
            raise ValueError(f"down must be experts x {W} x hidden, got {tuple(down.shape)}")
        E, _, F = down.shape
        rows = (2 if gated else 1) * F
        for name, t, shape, dtype in (("up", up, (E, rows, W), torch.int8), ("up_scale", up_scale, (E, rows), torch.float32),
                                      ("down", down, (E, W, F), torch.int8), ("down_scale", down_scale, (E, W), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {' x '.join(map(str, shape))} {dtype} tensor, got {t.dtype} {tuple(t.shape)}")
        with _on(stream, X, ids, weights, up, up_scale, down, down_scale):
            out = torch.empty(T, W, dtype=X.dtype, device=X.device)
            sgemm_expert_layer_int8(self.h, kind, int(gated), T, ids.shape[1], E, W, F, X, _ld(X), ids, weights, up, up_scale,
                                    down, down_scale, out, _ld(out))
        return out

    @property
    def last_variant(self):
        return sgemm_last_variant(self.h)

    def set_variant(self, v):
        sgemm_set_variant(self.h, v)

    def set_relayout(self, mode):
        sgemm_set_relayout(self.h, mode)

    @property
    def last_relayout(self) -> int:
        return sgemm_last_relayout(self.h)

    def device_status(self) -> int:
        return sgemm_get_device_status(self.h)

    def close(self):
        if self.h is not None:
            sgemm_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
