"""The int8 and expert calls on buffers past 2^31 elements or 2^32 bytes: rows at
the far end come out as rows at the near end do.  Expected values are computed
from the sampled rows alone (in 64 bits); tolerances as in test_gpu_int8.py and
test_gpu_experts.py."""
import numpy as np
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import plain_quantize

pytestmark = pytest.mark.gpu

V = sgemm
WIDTH = 8192
ROWS = (1 << 31) // WIDTH + 4099          # 2^31 elements and some: int8 offsets past 2^31, 16-bit ones past 2^32
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("too little free memory")
    h = sgemm.sgemm_create()
    yield h
    assert sgemm.sgemm_get_device_status(h) == V.OK
    sgemm.sgemm_destroy(h)
    torch.cuda.empty_cache()


def sampled():
    far = [ROWS - 1, ROWS - 2, (1 << 31) // WIDTH, (1 << 31) // WIDTH - 1, (1 << 30) // WIDTH + 7]
    return torch.tensor([0, 1, 12345] + far, device="cuda")


def test_product(handle):
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(-127, 128, (ROWS, WIDTH), dtype=torch.int8, device="cuda", generator=g)
    B = torch.randint(-127, 128, (72, WIDTH), dtype=torch.int8, device="cuda", generator=g)
    C = torch.zeros(ROWS, 72, device="cuda")
    one_a, one_b = torch.ones(ROWS, device="cuda"), torch.ones(72, device="cuda")
    at = sampled()
    want = (A[at].double() @ B.double().t()).float()
    for variant in (V.VARIANT_AUTO, V.VARIANT_GENERIC_I8):
        sgemm.sgemm_set_variant(handle, variant)
        C.zero_()
        sgemm.sgemm_run_int8(handle, 1, V.IN_F32, ROWS, 72, WIDTH, A, WIDTH, one_a, B, WIDTH, one_b, None, C, 72)
        torch.cuda.synchronize()
        assert torch.equal(C[at], want)
    sgemm.sgemm_set_variant(handle, V.VARIANT_AUTO)


def test_product_with_a_far_matrix(handle):
    """B_e past 2^31 elements, read in place and copied (K x N)."""
    E, N, K = 9, 1 << 15, WIDTH                      # 9 * 2^28 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    B = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    rows = 12
    A = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    off = torch.tensor([0] * E + [rows], dtype=torch.int32, device="cuda")   # all of the last expert
    C = torch.zeros(rows, N, device="cuda")
    sa, sb = torch.ones(rows, device="cuda"), torch.ones(E, N, device="cuda")
    sgemm.sgemm_run_int8_experts(handle, 1, V.IN_F32, E, rows, N, K, off, A, K, sa, B, K, N * K, sb, None, C, N)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 777, N - 2, N - 1], device="cuda")
    assert torch.equal(C[:, at], (A.double() @ B[E - 1][at].double().t()).float())


def test_quantize_and_moves(handle):
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(ROWS, WIDTH, dtype=torch.bfloat16, device="cuda", generator=g)
    Q, scale = torch.zeros(ROWS, WIDTH, dtype=torch.int8, device="cuda"), torch.zeros(ROWS, device="cuda")
    sgemm.sgemm_quantize_rows(handle, V.IN_BF16, ROWS, WIDTH, X, WIDTH, Q, WIDTH, scale)
    torch.cuda.synchronize()
    at = sampled()
    want_q, want_s = plain_quantize(X[at].cpu())
    assert np.array_equal(Q[at].cpu().numpy(), want_q) and np.array_equal(scale[at].cpu().numpy(), want_s)
    del Q

    # one choice a token, the tokens in reverse order
    rows = torch.arange(ROWS - 1, -1, -1, dtype=torch.int32, device="cuda")
    Y = torch.zeros_like(X)
    sgemm.sgemm_expert_dispatch(handle, V.IN_BF16, ROWS, 1, WIDTH, X, WIDTH, rows, Y, WIDTH)
    torch.cuda.synchronize()
    assert torch.equal(Y[ROWS - 1 - at], X[at])
    w = torch.rand(ROWS, device="cuda", generator=g)
    out = torch.zeros_like(X)
    sgemm.sgemm_expert_combine(handle, V.IN_BF16, ROWS, 1, WIDTH, Y, WIDTH, rows, w, out, WIDTH)
    dw, dY = torch.zeros(ROWS, device="cuda"), torch.zeros_like(X)
    sgemm.sgemm_expert_combine_grad(handle, V.IN_BF16, ROWS, 1, WIDTH, X, WIDTH, Y, WIDTH, rows, w, dY, WIDTH, dw)
    torch.cuda.synchronize()
    want = X[at].double() * w[at].double()[:, None]
    tol = (2 * EPS + 2.0 ** -8 * (1 + 2.0 ** -20)) * want.abs()
    assert bool(((out[at].double() - want).abs() <= tol).all())
    assert bool(((dY[ROWS - 1 - at].double() - want).abs() <= tol).all())
    square = X[at].double().square().sum(1)
    chain = WIDTH // 2048 * 8 + 5 + 8
    assert bool(((dw[at].double() - square).abs() <= 1.01 * chain * EPS * square).all())
