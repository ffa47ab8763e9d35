"""Scales over the whole range of E8M0, 2^-127 to 2^127: the largest, which other programs' buffers may
hold, make elements beyond FP32's largest number, but neither the product with a small scale nor with a
small row scale is one.

Products: the scales of a matrix are one power of two, so that sums of 32 to 300 products of two
codes, multiples of 2^-2 below 2^14, are exact.  Back: code times scale times row scale is rounded once."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests import fp4_util as f4
from tests.test_gpu_fp4 import check, Matrix, TYPES
from tests.test_gpu_fp4 import h, tile  # noqa: F401  (the handle; its reset)

pytestmark = pytest.mark.gpu

MX = sgemm.FP4_MX
PAIRS = [(0, 127), (127, 0), (0, 254), (254, 0), (253, 2), (252, 1), (254, 100), (60, 254), (0, 130), (130, 120)]


def rows_of(byte, row):
    def make(fmt, rows, K, gen):
        codes, scales, _ = f4.random_rows(fmt, rows, K, gen)
        return codes, torch.full_like(scales, byte), torch.full((rows,), row)
    return make


@pytest.mark.parametrize("variant", [sgemm.VARIANT_GENERIC_F4, sgemm.VARIANT_TC_F4, sgemm.VARIANT_TC_F4_PAIR])
@pytest.mark.parametrize("a,b", PAIRS)
@pytest.mark.parametrize("M,N,K", [(5, 70, 32), (70, 65, 33), (130, 130, 300)])
def test_products(h, tile, variant, a, b, M, N, K):  # noqa: F811
    sgemm.sgemm_set_variant(h, variant)

    def make(fmt, rows, K, gen):
        make.calls += 1
        return rows_of(a if make.calls % 2 else b, 1.0)(fmt, rows, K, gen)
    make.calls = 0
    check(h, MX, M, N, K, make=make, bias=False)
    assert sgemm.sgemm_last_variant(h)[0] == variant


@pytest.mark.parametrize("M,N,K", [(5, 70, 32), (70, 65, 100)])
def test_scales_of_both_ends_in_a_row(h, tile, M, N, K):  # noqa: F811
    """Blocks of 2^127 beside blocks of 2^-127, which meet their opposites: every variant the same sums."""
    def make(fmt, rows, K, gen):
        make.calls += 1
        codes, scales, row = f4.random_rows(fmt, rows, K, gen)
        at = torch.arange(scales.shape[1]) % 2 if make.calls % 2 else 1 - torch.arange(scales.shape[1]) % 2
        return codes, torch.where(at == 0, 254, 0).to(torch.uint8).expand_as(scales).contiguous(), row
    for variant in (sgemm.VARIANT_GENERIC_F4, sgemm.VARIANT_TC_F4, sgemm.VARIANT_TC_F4_PAIR):
        make.calls = 0
        sgemm.sgemm_set_variant(h, variant)
        check(h, MX, M, N, K, make=make, bias=False)


def test_a_nan_scale_in_the_generic_kernel(h, tile):  # noqa: F811
    """As on the tensor cores: NaN whatever its codes, zeros too, and no other row's."""
    sgemm.sgemm_set_variant(h, sgemm.VARIANT_GENERIC_F4)
    gen = torch.Generator().manual_seed(1)
    for which in (0, 1):
        parts = [f4.random_rows(MX, 70, 100, gen) for _ in range(2)]
        parts[which][0][3, 32:64] = 0
        parts[which][1][3, 1] = 255
        A, B = (Matrix(MX, 70, 100, gen, make=lambda *_, p=p: p) for p in parts)
        C = torch.full((70, 70), 7.0, device="cuda")
        sgemm.sgemm_run_fp4(h, MX, sgemm.IN_F32, 70, 70, 100, A.q, A.ld, A.s, None, B.q, B.ld, B.s, None, None, C, 70)
        c, want = C.cpu(), (A.values / A.row.cpu().double()[:, None]) @ (B.values / B.row.cpu().double()[:, None]).T
        nan = torch.zeros(70, 70, dtype=torch.bool)
        (nan if which == 0 else nan.T)[3] = True
        assert torch.equal(c.isnan(), nan) and torch.equal(c[~nan], want.float()[~nan])


@pytest.mark.parametrize("dtype", list(TYPES.values()))
@pytest.mark.parametrize("M,K", [(9, 33), (40, 4096), (7, 778)])
@pytest.mark.parametrize("row", [1.0, -1.0, 2.0 ** -20, 1.7e-38, 2.0 ** -126, 3e38, 0.0])
@pytest.mark.parametrize("byte", [0, 1, 100, 252, 253, 254])
def test_back(h, dtype, M, K, row, byte):  # noqa: F811
    kind = {v: k for k, v in TYPES.items()}[dtype]
    A = Matrix(MX, M, K, torch.Generator().manual_seed(byte), make=rows_of(byte, row))
    Y = torch.full((M, K), 7.0, dtype=dtype, device="cuda")
    sgemm.sgemm_dequantize_fp4(h, kind, MX, M, K, A.q, A.ld, A.s, A.row, Y, K)
    assert torch.equal(Y.cpu(), A.values.float().to(dtype))
