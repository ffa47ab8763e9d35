"""Host-side behaviour of the int8 and expert calls: argument checks, handle
checks and the marshalling of their arguments.  No GPU."""
import ctypes

import pytest

from dense_fp32_matrix_09_gb300 import build, sgemm

OK, NULL_, INVALID, ALIAS = sgemm.OK, sgemm.ERR_NULL, sgemm.ERR_INVALID_VALUE, sgemm.ERR_ALIAS
A0, B0, C0, SA, SB, BIAS, OFF = (0x10000000 * i for i in range(1, 8))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return sgemm.lib()


def chk(M=4, N=8, K=16, transB=1, out_type=sgemm.IN_F32, A=A0, lda=None, scaleA=SA, B=B0, ldb=None, scaleB=SB, bias=None,
        C=C0, ldc=None):
    return sgemm.sgemm_check_args_int8(transB, out_type, M, N, K, A, max(K, 1) if lda is None else lda, scaleA, B,
                                       max(K if transB else N, 1) if ldb is None else ldb, scaleB, bias, C,
                                       max(N, 1) if ldc is None else ldc)


def test_int8_sizes_and_enums():
    assert chk() == OK
    assert chk(transB=0) == OK
    assert chk(transB=0, ldb=7) == INVALID
    assert chk(ldb=15) == INVALID
    assert chk(lda=15) == INVALID
    assert chk(ldc=7) == INVALID
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(transB=2), dict(out_type=3), dict(out_type=-1)):
        assert chk(**bad) == INVALID, bad
    assert chk(K=131071) == OK              # 131071 * 2^14 < 2^31
    assert chk(K=131072) == INVALID
    for t in (sgemm.IN_F32, sgemm.IN_BF16, sgemm.IN_F16):
        assert chk(out_type=t) == OK


def test_int8_null_rules():
    assert chk(M=0, A=None, B=None, C=None, scaleA=None, scaleB=None) == OK
    assert chk(N=0, A=None, B=None, C=None, scaleA=None, scaleB=None) == OK
    assert chk(K=0, A=None, B=None) == OK
    for name in ("A", "B", "C", "scaleA", "scaleB"):
        assert chk(**{name: None}) == NULL_, name


def test_int8_alignment_rules():
    assert chk(A=A0 + 1, B=B0 + 3) == OK     # int8 operands: any address
    assert chk(C=C0 + 2) == INVALID
    assert chk(C=C0 + 2, out_type=sgemm.IN_F16) == OK
    assert chk(C=C0 + 1, out_type=sgemm.IN_F16) == INVALID
    for name in ("scaleA", "scaleB", "bias"):
        assert chk(**{name: SA + 2}) == INVALID, name


def test_int8_alias_rules():
    size = 3 * 8 * 4 + 8 * 4                                   # C's window: 4 x 8 FP32
    assert chk(C=A0) == ALIAS
    assert chk(C=B0 + 16 * 7 + 12) == ALIAS                    # inside B's last row
    assert chk(C=B0 + 16 * 8) == OK                            # just past it
    assert chk(C=SA - size) == OK
    assert chk(C=SA - size + 4) == ALIAS
    assert chk(bias=C0 + 8) == ALIAS
    assert chk(K=0, C=A0) == OK                                # A is not read


def test_int8_experts_rules():
    def ex(experts=3, rows=10, N=8, K=16, offsets=OFF, A=A0, B=B0, strideB=128, C=C0, bias=None):
        return sgemm.sgemm_check_args_int8_experts(1, sgemm.IN_BF16, experts, rows, N, K, offsets, A, 16, SA, B, 16,
                                                   strideB, SB, bias, C, 8)
    assert ex() == OK
    assert ex(strideB=0) == OK
    for bad in (dict(experts=0), dict(experts=1025), dict(strideB=-1), dict(rows=-1)):
        assert ex(**bad) == INVALID, bad
    assert ex(experts=1024) == OK
    assert ex(offsets=None) == NULL_
    assert ex(offsets=OFF + 1) == INVALID
    assert ex(C=B0 + 2 * 128 + 8) == ALIAS                     # inside the last expert's B
    assert ex(strideB=0, C=B0 + 2 * 128 + 8) == OK
    assert ex(C=OFF + 12) == ALIAS                             # the last of four offsets
    assert ex(C=OFF + 16) == OK


CALLS = [
    (sgemm.sgemm_run_int8, (1, 0, 4, 8, 16, A0, 16, SA, B0, 16, SB, None, C0, 8)),
    (sgemm.sgemm_run_int8_experts, (1, 0, 3, 4, 8, 16, OFF, A0, 16, SA, B0, 16, 1 << 40, SB, None, C0, 8)),
    (sgemm.sgemm_quantize_rows, (0, 4, 8, A0, 8, B0, 8, SA)),
    (sgemm.sgemm_expert_sort, (4, 2, 8, A0, B0, C0, SA)),
    (sgemm.sgemm_expert_dispatch, (0, 4, 2, 8, A0, 8, B0, C0, 8)),
    (sgemm.sgemm_expert_dispatch_int8, (0, 4, 2, 8, A0, 8, B0, C0, 8, SA)),
    (sgemm.sgemm_expert_dispatch_grad, (0, 4, 2, 8, A0, 8, B0, C0, 8)),
    (sgemm.sgemm_expert_combine, (0, 4, 2, 8, A0, 8, B0, SA, C0, 8)),
    (sgemm.sgemm_expert_combine_grad, (0, 4, 2, 8, A0, 8, B0, 8, C0, SA, SB, 8, BIAS)),
]


@pytest.mark.parametrize("call,args", CALLS, ids=[c.__name__ for c, _ in CALLS])
def test_bad_handles_are_rejected_without_dereference(call, args, monkeypatch):
    """Through the marshalling module and through ctypes alike."""
    assert sgemm.calls_module() is not None, build.calls_build_error
    for handle in (None, ctypes.c_void_p(0x1234)):
        with pytest.raises(sgemm.SgemmError) as e:
            call(handle, *args, stream=0)
        assert e.value.status == sgemm.ERR_BAD_HANDLE
    monkeypatch.setattr(sgemm, "_calls", None)
    monkeypatch.setattr(sgemm, "_calls_tried", True)
    with pytest.raises(sgemm.SgemmError) as e:
        call(None, *args, stream=0)
    assert e.value.status == sgemm.ERR_BAD_HANDLE


def test_marshalling_rejects_malformed_arguments():
    calls = sgemm.calls_module()
    assert calls is not None, build.calls_build_error
    good = CALLS[2][1]
    assert calls.enqueue("sgemm_quantize_rows", None, good, 0) == sgemm.ERR_BAD_HANDLE
    with pytest.raises(RuntimeError):
        calls.enqueue("sgemm_nothing", None, good, 0)
    with pytest.raises(TypeError):
        calls.enqueue("sgemm_quantize_rows", None, good[:-1], 0)
    with pytest.raises(TypeError):
        calls.enqueue("sgemm_quantize_rows", None, list(good), 0)
    with pytest.raises(OverflowError):
        calls.enqueue("sgemm_quantize_rows", None, (0, 1 << 40, *good[2:]), 0)
    with pytest.raises((TypeError, AttributeError)):
        calls.enqueue("sgemm_quantize_rows", None, (*good[:-1], object()), 0)


@pytest.mark.parametrize("call,args", CALLS, ids=[c.__name__ for c, _ in CALLS])
def test_numpy_integers_are_sizes_through_ctypes_too(call, args, monkeypatch):
    """Without the marshalling module the values that reach the library are the same."""
    import numpy as np
    real = getattr(sgemm.lib(), call.__name__)
    seen = []

    class Library:
        pass

    def record(*values):
        seen.append(tuple(v for v in values))
        return OK

    record.argtypes = real.argtypes
    library = Library()
    setattr(library, call.__name__, record)
    monkeypatch.setattr(sgemm, "_calls", None)
    monkeypatch.setattr(sgemm, "_calls_tried", True)
    monkeypatch.setattr(sgemm, "lib", lambda: library)
    call(None, *args, stream=0)
    sizes = [t is not ctypes.c_void_p for t in real.argtypes[1:-1]]
    call(None, *[np.int64(a) if s else a for a, s in zip(args, sizes)], stream=0)
    assert seen[0] == (None, *args, 0) and seen[1] == seen[0]
    assert all(type(v) is int or v is None for v in seen[1])
    with pytest.raises(TypeError):
        call(None, *[float(a) if s else a for a, s in zip(args, sizes)], stream=0)
    with pytest.raises(OverflowError):
        call(None, 1 << 40, *args[1:], stream=0)
    assert len(seen) == 2
