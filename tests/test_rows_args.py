"""Host-side behaviour of the norm, 4-bit and expert-layer calls: argument checks,
handle checks, the marshalling of their arguments, and what the tensor methods
refuse.  No GPU."""
import ctypes

import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm
from tests.test_tensor_methods import OnGpu

OK, NULL_, INVALID, ALIAS = sgemm.OK, sgemm.ERR_NULL, sgemm.ERR_INVALID_VALUE, sgemm.ERR_ALIAS
A0, B0, C0, SA, SB, RA, RB, BIAS = (0x10000000 * i for i in range(1, 9))
FORMATS = [sgemm.FP4_MX, sgemm.FP4_NV]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return sgemm.lib()


def chk(fmt=sgemm.FP4_NV, kind=sgemm.IN_F32, M=4, N=8, K=40, A=A0, lda=None, SA_=SA, RA_=RA, B=B0, ldb=None, SB_=SB, RB_=RB, bias=None, C=C0, ldc=None):
    wide = max((K + 1) // 2, 1)
    return sgemm.sgemm_check_args_fp4(fmt, kind, M, N, K, A, wide if lda is None else lda, SA_, RA_, B, wide if ldb is None else ldb, SB_, RB_, bias, C,
                                      max(N, 1) if ldc is None else ldc)


def test_scale_bytes():
    for fmt, block in ((sgemm.FP4_MX, 32), (sgemm.FP4_NV, 16)):
        for rows, K in ((1, 1), (128, 4 * block), (129, 4 * block), (5, 4 * block + 1), (0, 7), (7, 0), (1 << 30, 1 << 20)):
            words = -(-(-(-K // block)) // 4)
            assert sgemm.sgemm_fp4_scale_bytes(fmt, rows, K) == -(-rows // 128) * words * 512
    for bad in ((2, 1, 1), (-1, 1, 1), (0, -1, 1), (0, 1, -1), (0, (1 << 30) + 1, 1), (0, 1, (1 << 30) + 1)):
        assert sgemm.sgemm_fp4_scale_bytes(*bad) == -1, bad


def test_fp4_sizes_and_enums():
    for fmt in FORMATS:
        assert chk(fmt=fmt) == OK
        for K in (1, 2, 39, 41):
            assert chk(fmt=fmt, K=K) == OK
            for name in ("lda", "ldb"):
                assert chk(fmt=fmt, K=K, **{name: (K + 1) // 2 - 1}) == INVALID
    assert chk(ldc=7) == INVALID
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(fmt=2), dict(fmt=-1), dict(kind=3), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, ldc=1 << 31 >> 1)):
        assert chk(**bad) == INVALID, bad


def test_fp4_null_and_alignment_rules():
    assert chk(M=0, A=None, B=None, C=None, SA_=None, SB_=None, RA_=None, RB_=None) == OK
    assert chk(K=0, A=None, B=None, SA_=None, SB_=None) == OK
    assert chk(K=0, RA_=None) == NULL_
    for name in ("A", "B", "C", "SA_", "SB_", "RA_", "RB_"):
        assert chk(**{name: None}) == NULL_, name
    for name in ("RA_", "RB_"):
        assert chk(fmt=sgemm.FP4_MX, **{name: None}) == OK, name
    assert chk(A=A0 + 1, B=B0 + 3) == OK
    for name in ("SA_", "SB_"):
        assert chk(**{name: SA + 8}) == INVALID, name
    for name in ("RA_", "RB_", "bias", "C"):
        assert chk(**{name: BIAS + 2}) == INVALID, name


def test_fp4_alias_rules():
    size = 3 * 8 * 4 + 8 * 4
    for name, at, n in (("A", A0, 3 * 20 + 20), ("B", B0, 8 * 20), ("SA_", SA, 512), ("SB_", SB, 512), ("RA_", RA, 16), ("RB_", RB, 32)):
        assert chk(C=at) == ALIAS, name
        assert chk(C=at - size) == OK and chk(C=at - size + 4) == ALIAS, name
        assert chk(C=at + n) == OK and chk(C=at + n - 4) == ALIAS, name
    assert chk(C=BIAS, bias=BIAS) == ALIAS
    assert chk(C=A0, K=0) == OK


CALLS = {
    "sgemm_quantize_fp4": (0, 0, 4, 32, A0, 32, B0, 16, SA, None),
    "sgemm_dequantize_fp4": (0, 0, 4, 32, B0, 16, SA, None, A0, 32),
    "sgemm_run_fp4": (0, 0, 4, 8, 32, A0, 16, SA, None, B0, 16, SB, None, None, C0, 8),
    "sgemm_rms_norm": (0, 4, 32, A0, 32, None, 0, B0, 1e-5, None, 0, C0, 32, None),
    "sgemm_rms_norm_int8": (0, 4, 32, A0, 32, None, 0, B0, 1e-5, None, 0, C0, 32, SA),
    "sgemm_rms_norm_fp4": (0, 0, 4, 32, A0, 32, None, 0, B0, 1e-5, None, 0, C0, 16, SA, SB),
    "sgemm_rms_norm_grad": (0, 4, 32, A0, 32, None, 0, B0, 32, C0, SA, SB, 32, RA),
    "sgemm_expert_layer_int8": (0, 1, 4, 2, 3, 32, 16, A0, 32, B0, C0, SA, SB, RA, RB, BIAS, 32),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_handles_come_first(name):
    with pytest.raises(sgemm.SgemmError) as e:
        getattr(sgemm, name)(None, *CALLS[name], stream=0)
    assert e.value.status == sgemm.ERR_BAD_HANDLE
    with pytest.raises(sgemm.SgemmError) as e:
        getattr(sgemm, name)(ctypes.c_void_p(0x1234), *CALLS[name], stream=0)
    assert e.value.status == sgemm.ERR_BAD_HANDLE


@pytest.mark.parametrize("name", list(CALLS))
def test_marshalled_as_declared(name):
    """The compiled marshalling has as many arguments, of the same kinds, as the binding declares."""
    calls = sgemm.calls_module()
    assert calls is not None, build.calls_build_error
    kinds = getattr(sgemm.lib(), name).argtypes[1:-1]
    assert len(kinds) == len(CALLS[name])
    assert calls.enqueue(name, None, CALLS[name], 0) == sgemm.ERR_BAD_HANDLE
    with pytest.raises(TypeError):
        calls.enqueue(name, None, CALLS[name][:-1], 0)
    for i, kind in enumerate(kinds):
        wrong = {ctypes.c_int: 1 << 40, ctypes.c_float: "x", ctypes.c_void_p: object()}[kind]
        with pytest.raises((OverflowError, TypeError, AttributeError)):
            calls.enqueue(name, None, (*CALLS[name][:i], wrong, *CALLS[name][i + 1:]), 0)


# ---- the tensor methods -----------------------------------------------------------------
T, K, N, E, F, J = 4, 32, 8, 3, 16, 2


def fp4(rows, k=K, fmt=sgemm.FP4_NV, **change):
    parts = dict(Q=torch.zeros(rows, 16, dtype=torch.uint8), S=torch.zeros(sgemm.sgemm_fp4_scale_bytes(fmt, rows, k), dtype=torch.uint8), row=torch.ones(rows))
    return {**parts, **change}


def arguments():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    x = lambda: torch.zeros(T, K)  # noqa: E731
    return {
        "quantize_fp4": dict(X=x()),
        "dequantize_fp4": dict(A=fp4(T), out=x()),
        "matmul_fp4": dict(A=fp4(T), B=fp4(N), bias=torch.ones(N), out=torch.zeros(T, N)),
        "rms_norm": dict(X=x(), weight=torch.ones(K), residual=x()),
        "rms_norm_int8": dict(X=x(), weight=torch.ones(K), residual=x()),
        "rms_norm_fp4": dict(X=x(), weight=torch.ones(K), residual=x()),
        "rms_norm_grad": dict(dY=x(), H=x(), weight=torch.ones(K), rstd=torch.ones(T), dH=x()),
        "expert_layer_int8": dict(X=x(), ids=torch.zeros(T, J, dtype=torch.int32), weights=torch.ones(T, J), up=i8(E, F, K), up_scale=torch.ones(E, F),
                                  down=i8(E, K, F), down_scale=torch.ones(E, K)),
    }


def leaves():
    for m, args in arguments().items():
        for a, v in args.items():
            yield from ((m, a, part) for part in v) if isinstance(v, dict) else [(m, a, None)]


@pytest.fixture
def g(monkeypatch):
    def reached(*args, **kwargs):
        raise AssertionError("the library was called")
    monkeypatch.setattr(sgemm, "_enqueue", reached)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    g = object.__new__(sgemm.Sgemm)
    g.h = None
    return g


def call(g, method, name, part, make):
    """The method with every tensor on the GPU but the named one, which `make` gives."""
    def value(a, p, t):
        return make(t) if (a, p) == (name, part) else OnGpu(t)
    args = {a: sgemm.Fp4Rows(**{p: value(a, p, t) for p, t in v.items()}, K=K, format=sgemm.FP4_NV) if isinstance(v, dict) else value(a, None, v)
            for a, v in arguments()[method].items()}
    getattr(g, method)(**args)


@pytest.mark.parametrize("method,name,part", list(leaves()))
def test_a_tensor_elsewhere_is_refused(g, method, name, part):
    with pytest.raises(ValueError, match="must be on the GPU"):
        call(g, method, name, part, lambda t: t)
    with pytest.raises(ValueError, match="must be on the current device"):
        call(g, method, name, part, lambda t: OnGpu(t, 1))


WRONG = [("dequantize_fp4", "A", "Q", torch.zeros(T, 15, dtype=torch.uint8)), ("dequantize_fp4", "A", "Q", torch.zeros(T, 16)),
         ("matmul_fp4", "A", "S", torch.zeros(511, dtype=torch.uint8)), ("matmul_fp4", "B", "row", torch.ones(N + 1)), ("matmul_fp4", "bias", None, torch.ones(N + 1)),
         ("matmul_fp4", "out", None, torch.zeros(T, N + 1)), ("rms_norm", "weight", None, torch.ones(K + 1)), ("rms_norm", "weight", None, torch.ones(K).bfloat16()),
         ("rms_norm_int8", "residual", None, torch.zeros(T, K + 1)), ("rms_norm_fp4", "residual", None, torch.zeros(T, K).half()),
         ("rms_norm_grad", "rstd", None, torch.ones(T + 1)), ("rms_norm_grad", "dY", None, torch.zeros(T, K).half()), ("rms_norm_grad", "dH", None, torch.zeros(T + 1, K)),
         ("quantize_fp4", "X", None, torch.zeros(T, K).double()), ("expert_layer_int8", "ids", None, torch.zeros(T, J, dtype=torch.int64)),
         ("expert_layer_int8", "up", None, torch.zeros(E, F + 1, K, dtype=torch.int8)), ("expert_layer_int8", "down", None, torch.zeros(E, K, F)),
         ("expert_layer_int8", "weights", None, torch.ones(T, J + 1)), ("expert_layer_int8", "down_scale", None, torch.ones(E, K + 1))]


@pytest.mark.parametrize("method,name,part,value", WRONG, ids=[f"{m}-{n}-{i}" for i, (m, n, _, _) in enumerate(WRONG)])
def test_wrong_shapes_and_types_are_refused(g, method, name, part, value):
    with pytest.raises(ValueError):
        call(g, method, name, part, lambda t: OnGpu(value))


def test_rows_that_do_not_fit_together_are_refused(g):
    gpu = lambda fmt, k, **c: sgemm.Fp4Rows(**{p: None if t is None else OnGpu(t) for p, t in fp4(T, k, fmt, **c).items()}, K=k, format=fmt)  # noqa: E731
    for a, b in ((gpu(0, K), gpu(1, K)), (gpu(1, K), gpu(1, K - 1)), (gpu(1, K, row=None), gpu(1, K)), (gpu(1, K), gpu(1, K)._replace(format=5)),
                 (gpu(0, 33), gpu(0, 33))):
        with pytest.raises(ValueError):
            g.matmul_fp4(a, b)


def test_tiled_scales():
    from tests import fp4_util as f4
    for fmt in FORMATS:
        for rows, k in ((1, 1), (130, 300), (33, 64)):
            s = torch.randint(0, 255, (rows, sgemm.fp4_blocks(fmt, k)), dtype=torch.uint8)
            t = sgemm.fp4_tile_scales(s, fmt, k)
            assert t.numel() == sgemm.sgemm_fp4_scale_bytes(fmt, rows, k) and torch.equal(t, f4.tiled(fmt, s, k))
            assert torch.equal(t[f4.scale_index(fmt, rows, k).reshape(-1)].view(s.shape), s)
        with pytest.raises(ValueError):
            sgemm.fp4_tile_scales(torch.zeros(3, 5, dtype=torch.uint8), fmt, 32)
