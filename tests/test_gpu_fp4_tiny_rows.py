"""Rows of tiny values to 4 bits of format NV: the quotient (2688 / m) / s passes FP32's range
below m = 2688 * 2^-119 for the smallest scales s.

The definition does not change when a row is multiplied by a power of two (with an exponent
without bounds, as it says), and 2^16 times larger these rows are far from any bound: their
codes and scales must be those of the larger rows, bit for bit, and the row scales m / 2688."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests import fp4_util as f4
from tests.test_gpu_fp4 import quantized, same_codes
from tests.test_gpu_fp4 import h  # noqa: F401  (the handle)

pytestmark = pytest.mark.gpu

NV = sgemm.FP4_NV
LIFT = 2.0 ** 16
TYPES = {torch.float32: sgemm.IN_F32, torch.bfloat16: sgemm.IN_BF16}  # (FP16 has no such values)
# from just above the rows that are stored as zeros to well past the bound
MAXIMA = [3.2e-35, 3.3e-35, 1e-34, 7.7e-34, 2688 * 2.0 ** -119, 4.1e-33, 2688 * 2.0 ** -118, 9e-33, 1e-32, 1e-31]


def tiny_rows(K, dtype, seed=0):
    """A row for each of MAXIMA whose blocks are 1 to 1e5 times smaller, with zeros of both signs among them."""
    gen = torch.Generator().manual_seed(K + seed)
    x = torch.randn(len(MAXIMA), K, generator=gen, dtype=torch.float64)
    x /= x.abs().amax(dim=1, keepdim=True)
    size = 10.0 ** -(torch.arange(f4.blocks_of(NV, K)) % 11 / 2.0)
    x *= size.repeat_interleave(16)[:K]
    x[:, 3::5] = 0
    x[:, 4::10] = -0.0
    x[:, 0] = 1
    return (x * torch.tensor(MAXIMA, dtype=torch.float64)[:, None]).to(dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K", [17, 33, 145, 160, 777, 4096, 20001])
def test_quantize(h, dtype, K):  # noqa: F811
    x = tiny_rows(K, dtype)
    codes, scales, _ = f4.quantize(NV, x.double() * LIFT)
    assert ((codes & 7)[x == 0] == 0).all() and (scales > 0).any(dim=1).all()
    for more in (dict(), dict(ldx=K + 3, pad=2), dict(off=1)):
        got, s, row, _ = quantized(h, NV, x, **more)
        assert torch.equal(s, scales)
        assert same_codes(got, codes)
        assert torch.equal(row, x.float().abs().amax(dim=1) / torch.tensor(2688.0))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_there_and_back(h, dtype):  # noqa: F811
    """Back in FP32: code times scale is exact, times the row's rounded once (row scales from 2^-126 on, so that
    a product may be subnormal: half a unit of those, 2^-150, at most)."""
    K = 401
    x = tiny_rows(K, dtype, 1)
    codes, scales, row, (Q, S, r, ld) = quantized(h, NV, x)
    Y = torch.full((len(x), K), 7.0, device="cuda")
    sgemm.sgemm_dequantize_fp4(h, sgemm.IN_F32, NV, len(x), K, Q, ld, S, r, Y, K)
    y = Y.cpu().double()
    assert ((y - f4.values(NV, codes, scales, row)).abs() <= 2.0 ** -24 * y.abs() + 2.0 ** -150).all()
    assert (y[x == 0] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K", [145, 640])
def test_norm(h, dtype, K):  # noqa: F811
    """Rows of ordinary size and weights so small that what is quantized falls into the range."""
    w, M = tiny_rows(K, dtype)[2], 5
    gen = torch.Generator().manual_seed(K)
    x = (torch.randn(M, K, generator=gen).abs() + 0.5).to(dtype)
    v = x.float() * w.float()
    codes, scales, m = f4.quantize(NV, v.double() * LIFT)
    X, W = x.cuda(), w.cuda()
    wide = (K + 1) // 2
    Q = torch.zeros(M, wide, dtype=torch.uint8, device="cuda")
    S = torch.zeros(sgemm.sgemm_fp4_scale_bytes(NV, M, K), dtype=torch.uint8, device="cuda")
    row = torch.zeros(M, device="cuda")
    sgemm.sgemm_rms_norm_fp4(h, TYPES[dtype], NV, M, K, X, K, None, 0, W, 1e-5, None, 0, Q, wide, S, row)
    assert torch.equal(S.cpu(), f4.tiled(NV, scales, K))
    assert same_codes(f4.unpack(Q.cpu(), K), codes)
    rstd = 1 / torch.sqrt(x.double().square().mean(dim=1) + 1e-5)
    want = v.double().abs().amax(dim=1) / 2688 * rstd
    assert ((row.cpu().double() - want).abs() <= (53 / 2 + 6) * 2.0 ** -24 * want + 2.0 ** -149).all()
