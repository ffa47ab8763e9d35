"""The norm with eps = 0: a row of zeros has r = infinity.  Its Y is what the formula says,
0 times infinity, a NaN; quantized it is the row of zeros that the quantizers make of one."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests import fp4_util as f4
from tests.test_gpu_norm import KINDS, U, chain, rows
from tests.test_gpu_norm import h  # noqa: F401  (the handle)

pytestmark = pytest.mark.gpu


def problem(dtype, K):
    gen = torch.Generator().manual_seed(K)
    x, w = rows(7, K, gen, dtype), (1 + 0.3 * torch.randn(K, generator=gen)).to(dtype)
    x[5] = -0.0
    zero = torch.tensor([False, False, True, False, False, True, False])   # (rows makes the third one zero)
    assert torch.equal((x == 0).all(dim=1), zero)
    return x, w, zero, 1 / torch.sqrt(x.double().square().mean(dim=1))


@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("K", [1, 33, 640, 20000])
def test_own_type_and_8_bits(h, dtype, K):  # noqa: F811
    x, w, zero, r = problem(dtype, K)
    X, W, Y, rstd = x.cuda(), w.cuda(), torch.zeros_like(x).cuda(), torch.zeros(7, device="cuda")
    sgemm.sgemm_rms_norm(h, KINDS[dtype], 7, K, X, K, None, 0, W, 0.0, None, 0, Y, K, rstd)
    y, got = Y.cpu(), rstd.cpu()
    assert got[zero].isinf().all() and y[zero].isnan().all() and y[~zero].isfinite().all()
    assert ((got.double() - r)[~zero].abs() <= (chain(K) / 2 + 4) * U * r[~zero]).all()
    Q, scale = torch.ones(7, K, dtype=torch.int8, device="cuda"), torch.ones(7, device="cuda")
    sgemm.sgemm_rms_norm_int8(h, KINDS[dtype], 7, K, X, K, None, 0, W, 0.0, None, 0, Q, K, scale)
    assert (Q.cpu()[zero] == 0).all() and (scale.cpu()[zero] == 0).all() and scale.isfinite().all()


@pytest.mark.parametrize("fmt", [sgemm.FP4_MX, sgemm.FP4_NV])
@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("K", [1, 33, 640, 20000])
def test_4_bits(h, fmt, dtype, K):  # noqa: F811
    x, w, zero, r = problem(dtype, K)
    X, W, wide = x.cuda(), w.cuda(), (K + 1) // 2
    Q = torch.full((7, wide), 0x77, dtype=torch.uint8, device="cuda")
    S = torch.zeros(sgemm.sgemm_fp4_scale_bytes(fmt, 7, K), dtype=torch.uint8, device="cuda")
    row = torch.ones(7, device="cuda")
    sgemm.sgemm_rms_norm_fp4(h, KINDS[dtype], fmt, 7, K, X, K, None, 0, W, 0.0, None, 0, Q, wide, S, row)
    codes, scales, m = f4.quantize(fmt, x.float() * w.float())
    assert torch.equal(f4.code_values(f4.unpack(Q.cpu(), K)), f4.code_values(codes))
    assert torch.equal(S.cpu(), f4.tiled(fmt, scales, K))
    got, want = row.cpu(), r if fmt == sgemm.FP4_MX else m.double() / 2688 * r
    assert (got[zero] == 0).all()
    assert ((got.double() - want)[~zero].abs() <= (chain(K) / 2 + 6) * U * want[~zero]).all()
    # and a product of them: zeros for the rows of zeros, no NaN anywhere
    b = torch.ones(5, K).to(dtype).cuda()
    qb, sb, rb = torch.zeros(5, wide, dtype=torch.uint8, device="cuda"), torch.zeros_like(S), torch.ones(5, device="cuda")
    sgemm.sgemm_quantize_fp4(h, KINDS[dtype], fmt, 5, K, b, K, qb, wide, sb, rb)
    C = torch.full((7, 5), 9.0, device="cuda")
    sgemm.sgemm_run_fp4(h, fmt, sgemm.IN_F32, 7, 5, K, Q, wide, S, row, qb, wide, sb, rb, None, C, 5)
    c = C.cpu()
    assert c.isfinite().all() and (c[zero] == 0).all()
