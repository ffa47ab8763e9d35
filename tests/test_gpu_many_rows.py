"""The routing and quantization calls at their most rows: indices that pass 2^31
when a grid's step is added to them, and block counts near it.  One element a
row and one choice a token, so that every expected value is one exact or
correctly rounded FP32 operation, rounded once more to FP16: results are equal."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm

pytestmark = pytest.mark.gpu

V = sgemm
MOST = 2 ** 31 - 1                # rows: what the calls accept
OVER = 2 ** 30 + 4099             # twice this many passes 2^31
PART = 1 << 28


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("too little free memory")
    h = sgemm.sgemm_create()
    yield h
    assert sgemm.sgemm_get_device_status(h) == V.OK
    sgemm.sgemm_destroy(h)
    torch.cuda.empty_cache()


def halves(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(n, dtype=torch.float16, device="cuda")
    for i in range(0, n, PART):
        m = min(PART, n - i)
        x[i:i + m] = torch.randn(m, generator=g, device="cuda")
    return x


def parts(n):
    return [(i, min(i + PART, n)) for i in range(0, n, PART)]


def backwards(n):
    return torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")


def test_dispatch(handle):
    X, Y = halves(MOST, 1), torch.zeros(MOST, dtype=torch.float16, device="cuda")
    sgemm.sgemm_expert_dispatch(handle, V.IN_F16, MOST, 1, 1, X, 1, backwards(MOST), Y, 1)
    torch.cuda.synchronize()
    for i, j in parts(MOST):
        assert torch.equal(Y[MOST - j:MOST - i].flip(0), X[i:j])


def test_combine(handle):
    Y, out = halves(MOST, 2), torch.zeros(MOST, dtype=torch.float16, device="cuda")
    w = torch.empty(MOST, device="cuda")
    for i, j in parts(MOST):
        w[i:j] = (torch.arange(i, j, device="cuda") % 1021).float() / 1021
    sgemm.sgemm_expert_combine(handle, V.IN_F16, MOST, 1, 1, Y, 1, backwards(MOST), w, out, 1)
    torch.cuda.synchronize()
    for i, j in parts(MOST):
        assert torch.equal(out[i:j], (w[i:j] * Y[MOST - j:MOST - i].flip(0).float()).half())


@pytest.mark.parametrize("n", [OVER, MOST])
def test_combine_gradients(handle, n):
    dout, Y, dY = halves(n, 3), halves(n, 4), torch.zeros(n, dtype=torch.float16, device="cuda")
    w, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    for i, j in parts(n):
        w[i:j] = (torch.arange(i, j, device="cuda") % 1021).float() / 1021
    sgemm.sgemm_expert_combine_grad(handle, V.IN_F16, n, 1, 1, dout, 1, Y, 1, backwards(n), w, dY, 1, dw)
    torch.cuda.synchronize()
    for i, j in parts(n):
        g = dout[i:j].float()
        assert torch.equal(dY[n - j:n - i].flip(0), (w[i:j] * g).half())
        assert torch.equal(dw[i:j], g * Y[n - j:n - i].flip(0).float())


def test_quantize(handle):
    X = halves(MOST, 5)
    Q, scale = torch.zeros(MOST, dtype=torch.int8, device="cuda"), torch.full((MOST,), -1.0, device="cuda")
    sgemm.sgemm_quantize_rows(handle, V.IN_F16, MOST, 1, X, 1, Q, 1, scale)
    torch.cuda.synchronize()
    steps = torch.full((1,), 127.0, device="cuda")      # (a division by a tensor is a division)
    for i, j in parts(MOST):
        x = X[i:j].float()
        assert torch.equal(Q[i:j], (127 * x.sign()).to(torch.int8))
        assert torch.equal(scale[i:j], x.abs() / steps)
