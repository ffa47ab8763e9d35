"""The quantization and routing kernels' further forms, which the number of rows
and their width choose: a warp or a block a token, one to four pieces of a row a
thread, several pieces in turn, every width of access.

Tolerances as in test_gpu_experts.py, but for the longest chain of a dot product,
which depends on the form: with a warp a token a thread takes 8 of every 256
elements and 5 steps follow within the warp; with a block 8 of every 2048, 5
steps and 8 warps."""
import numpy as np
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_experts import EPS, Routed, handle  # noqa: F401  (fixture)
from tests.test_gpu_int8 import TYPES, addr, plain_quantize, strided

pytestmark = pytest.mark.gpu

V = sgemm


def chain(tokens, width):
    if width < 2048 and tokens >= width // 2:           # a warp a token
        return -(-width // 256) * 8 + 5
    return -(-width // 2048) * 8 + 5 + 8


def token_sums(values, kept, choices, tokens):
    """Sums of the kept slots' rows by token, and of their magnitudes."""
    want, mag = (np.zeros((tokens, values.shape[1])) for _ in range(2))
    np.add.at(want, kept // choices, values)
    np.add.at(mag, kept // choices, np.abs(values))
    return want, mag


# a warp a token (width < 2048, tokens >= width / 2) and, at the same widths, a block
NARROW = [(300, 2, 512), (700, 4, 1000), (600, 9, 257), (1100, 1, 2047), (1024, 3, 2040), (130, 5, 256), (64, 2, 128),
          (40, 7, 72), (513, 2, 1024)]
BLOCK = [(299, 2, 600), (100, 4, 1000), (120, 9, 257), (20, 3, 2047), (700, 2, 2048), (5, 2, 1024)]
LAYOUTS = [(0, 0), (8, 8), (4, 4), (2, 2), (1, 3)]       # accesses of 16, 16, 8 (FP32: 16), 4 (8) bytes, one element


@pytest.mark.parametrize("tokens,choices,width", NARROW + BLOCK)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", LAYOUTS)
def test_combine_and_its_gradients(handle, tokens, choices, width, dtype, pad, offset):  # noqa: F811
    t = Routed(handle, tokens, choices, width, dtype, pad, offset)
    y, out, dout, dy = t.buf(t.slots), t.buf(tokens, 9.0), t.buf(tokens), t.buf(t.slots, 9.0)
    unused = np.setdiff1d(np.arange(t.slots), t.r[t.kept])
    y[0][torch.as_tensor(unused, device="cuda")] = float("nan")
    w = torch.rand(tokens, choices, generator=t.g)
    w.view(-1)[np.setdiff1d(np.arange(t.slots), t.kept)] = float("nan")
    W, dw = w.cuda(), torch.full((t.slots + 1,), -7.0, device="cuda")
    sgemm.sgemm_expert_combine(handle, t.kind, tokens, choices, width, t.p(y), t.ld, t.rows, W, t.p(out), t.ld)
    sgemm.sgemm_expert_combine_grad(handle, t.kind, tokens, choices, width, t.p(dout), t.ld, t.p(y), t.ld, t.rows, W,
                                    t.p(dy), t.ld, dw)
    torch.cuda.synchronize()
    mine, token = t.r[t.kept], t.kept // choices
    yd, gd, wd = t.double(y)[mine], t.double(dout)[token], w.double().numpy().reshape(-1)[t.kept, None]
    want, mag = token_sums(wd * yd, t.kept, choices, tokens)
    assert np.all(np.abs(t.double(out) - want) <= 1.01 * choices * EPS * mag + t.u * np.abs(want) * (1 + 2.0 ** -20) + t.tiny)
    t.untouched(out, 9.0, np.arange(tokens))
    want_dw, mag_dw = np.zeros(t.slots), np.zeros(t.slots)
    want_dw[t.kept], mag_dw[t.kept] = (gd * yd).sum(1), np.abs(gd * yd).sum(1)
    assert np.all(np.abs(dw[:-1].cpu().double().numpy() - want_dw) <= 1.01 * chain(tokens, width) * EPS * mag_dw)
    assert float(dw[-1]) == -7.0
    got_dy, want_dy = t.double(dy)[mine], wd * gd
    assert np.all(np.abs(got_dy - want_dy) <= (EPS + t.u * (1 + 2.0 ** -20)) * np.abs(want_dy) + t.tiny)
    t.untouched(dy, 9.0, mine)


@pytest.mark.parametrize("tokens,choices,width", [(300, 2, 512), (700, 4, 1000), (600, 9, 257), (1100, 1, 2047), (900, 4, 96),
                                                  (700, 2, 4096)])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", LAYOUTS)
def test_dispatch_and_its_gradient(handle, tokens, choices, width, dtype, pad, offset):  # noqa: F811
    t = Routed(handle, tokens, choices, width, dtype, pad, offset)
    x, y, dy, dx = t.buf(tokens), t.buf(t.slots, 9.0), t.buf(t.slots), t.buf(tokens, 9.0)
    dy[0][torch.as_tensor(np.setdiff1d(np.arange(t.slots), t.r[t.kept]), device="cuda")] = float("nan")
    sgemm.sgemm_expert_dispatch(handle, t.kind, tokens, choices, width, t.p(x), t.ld, t.rows, t.p(y), t.ld)
    sgemm.sgemm_expert_dispatch_grad(handle, t.kind, tokens, choices, width, t.p(dy), t.ld, t.rows, t.p(dx), t.ld)
    torch.cuda.synchronize()
    assert torch.equal(y[0].cpu()[t.r[t.kept]], x[0].cpu()[t.kept // choices])
    t.untouched(y, 9.0, t.r[t.kept])
    want, mag = token_sums(t.double(dy)[t.r[t.kept]], t.kept, choices, tokens)
    assert np.all(np.abs(t.double(dx) - want) <= 1.01 * choices * EPS * mag + t.u * np.abs(want) * (1 + 2.0 ** -20) + t.tiny)
    t.untouched(dx, 9.0, np.arange(tokens))


# more than four rows an SM: 32 to 512 threads a row by its width, one piece of 8 elements
# a thread, four of them, or more than the registers hold
WIDTHS = [5, 200, 256, 257, 700, 1000, 1024, 1025, 1500, 2048, 2049, 3000, 4096, 4097, 5000, 8190, 8192, 8193, 16384, 16400]


def rows_with_outliers(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))
    x[torch.arange(M), torch.randint(0, K, (M,), generator=g)] *= 20     # the largest anywhere in the row
    x[1] = 0
    x[2, K - 1] = float("inf")
    x[3, K // 2] = float("nan")
    return x.to(TYPES[dtype][1])


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
def test_quantize_many_rows(handle, K, dtype, pad, offset):  # noqa: F811
    M = 900
    x = rows_with_outliers(M, K, dtype, K)
    X, Xf = strided(x, pad, offset, fill=1.0e4)
    Q, Qf = strided(torch.full((M, K), 99, dtype=torch.int8), pad, offset, fill=99)
    scale = torch.full((M + 1,), -1.0, device="cuda")
    sgemm.sgemm_quantize_rows(handle, TYPES[dtype][0], M, K, addr(X, Xf, offset), K + pad, addr(Q, Qf, offset), K + pad,
                              scale)
    torch.cuda.synchronize()
    want_q, want_s = plain_quantize(x)
    assert np.array_equal(scale[:M].cpu().numpy(), want_s, equal_nan=True) and float(scale[M]) == -1.0
    assert np.array_equal(Q.cpu().numpy(), want_q)
    Q.fill_(99)
    assert bool((Qf == 99).all())


@pytest.mark.parametrize("tokens,choices,width", [(700, 2, 1000), (700, 4, 4096), (650, 3, 2050), (2000, 2, 512), (620, 1, 8200)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_dispatch_int8_of_a_prompt(handle, tokens, choices, width, dtype):  # noqa: F811
    t = Routed(handle, tokens, choices, width, dtype, 0, 0)
    x = rows_with_outliers(tokens, width, dtype, width)
    q, qf = strided(torch.full((t.slots, width), 99, dtype=torch.int8), 0, 0, fill=99)
    scale = torch.full((t.slots + 1,), -1.0, device="cuda")
    sgemm.sgemm_expert_dispatch_int8(handle, t.kind, tokens, choices, width, x.cuda(), width, t.rows, q, width, scale)
    torch.cuda.synchronize()
    want_q, want_s = plain_quantize(x)
    got_q, got_s = q.cpu().numpy(), scale.cpu().numpy()
    mine, token = t.r[t.kept], t.kept // choices
    assert np.array_equal(got_q[mine], want_q[token])
    assert np.array_equal(got_s[mine], want_s[token], equal_nan=True)
    rest = np.setdiff1d(np.arange(t.slots), mine)
    assert np.all(got_q[rest] == 99) and np.all(got_s[rest] == -1) and got_s[-1] == -1
    assert bool((qf[t.slots * width:] == 99).all())
