"""4-bit rows and their products on the GPU.

The products are checked bit for bit: with every code, and scales that are powers of
two near 1, each product is a multiple of 2^-4 (codes 1/2 * 1/2, scales 1/2 * 1/2) and every
partial sum stays below 2^20, so FP32 sums are exact in any order and whatever they
are truncated to.  Random data in general is then held to a bound that counts one
truncation (2^-23 of the terms' magnitudes) a product."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm
from tests import fp4_util as f4

pytestmark = pytest.mark.gpu

FORMATS = [sgemm.FP4_MX, sgemm.FP4_NV]
TYPES = {sgemm.IN_F32: torch.float32, sgemm.IN_BF16: torch.bfloat16, sgemm.IN_F16: torch.float16}


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    h = sgemm.sgemm_create()
    yield h
    torch.cuda.synchronize()
    assert sgemm.sgemm_get_device_status(h) == sgemm.OK
    sgemm.sgemm_destroy(h)


class Matrix:
    """A random matrix in 4 bits on the GPU; `shift` bytes off a 16-byte boundary, `pad` more a row."""

    def __init__(self, fmt, rows, K, gen, shift=0, pad=None, make=None):
        codes, scales, row = (make or f4.random_rows)(fmt, rows, K, gen)
        wide = (K + 1) // 2
        self.ld = -(-wide // 16) * 16 if pad is None else wide + pad
        host = torch.full((shift + rows * self.ld + 64,), 0xEE, dtype=torch.uint8)
        body = host[shift:shift + rows * self.ld].view(rows, self.ld)
        body[:, :wide] = f4.pack(codes)
        self.buf = host.cuda()
        self.q = self.buf.data_ptr() + shift
        self.s = f4.tiled(fmt, scales, K, fill=0x7f if fmt == sgemm.FP4_NV else 0xff).cuda()  # NaN behind the last row
        self.row = row.cuda()
        self.values = f4.values(fmt, codes, scales, row)


def product(h, fmt, M, N, K, kind=sgemm.IN_F32, bias=True, seed=0, a=None, b=None, rows=True, ldc=None, make=None):
    gen = torch.Generator().manual_seed(1000 * seed + 7 * M + 3 * N + K)
    A, B = Matrix(fmt, M, K, gen, make=make, **(a or {})), Matrix(fmt, N, K, gen, make=make, **(b or {}))
    bias_t = torch.randint(-8, 9, (N,), generator=gen).float() / 4 if bias else None
    ldc = ldc or N
    C = torch.full((M + 1, ldc), 77.0, dtype=TYPES[kind], device="cuda")
    dbias = None if bias_t is None else bias_t.cuda()
    sgemm.sgemm_run_fp4(h, fmt, kind, M, N, K, A.q, A.ld, A.s, A.row if rows else None, B.q, B.ld, B.s, B.row if rows else None, dbias, C, ldc)
    torch.cuda.synchronize()
    assert sgemm.sgemm_get_device_status(h) == sgemm.OK
    got = C.cpu()
    assert (got[M] == 77).all() and (got[:M, N:] == 77).all()
    va, vb = (A.values, B.values) if rows else (A.values / A.row.cpu().double()[:, None], B.values / B.row.cpu().double()[:, None])
    want = va @ vb.T
    if bias:
        want = want + bias_t.double()
    return got[:M, :N], want, va.abs() @ vb.abs().T


def check(h, fmt, M, N, K, kind=sgemm.IN_F32, **more):
    got, want, _ = product(h, fmt, M, N, K, kind, **more)
    want = want.float().to(TYPES[kind])
    bad = (got != want).nonzero()
    assert not len(bad), f"{len(bad)} of {got.numel()} differ, first at {bad[0].tolist()}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


@pytest.fixture
def tile(h):
    def pin(tokens, split):
        sgemm.sgemm_debug_set_fp4_tile(h, tokens, split)
    yield pin
    sgemm.sgemm_debug_set_fp4_tile(h, 0, 0)
    sgemm.sgemm_set_variant(h, sgemm.VARIANT_AUTO)
    sgemm.sgemm_set_relayout(h, sgemm.RELAYOUT_AUTO)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 15), (2, 130, 64), (17, 257, 300), (70, 65, 33), (130, 64, 1000)])
def test_generic(h, tile, fmt, M, N, K):
    sgemm.sgemm_set_variant(h, sgemm.VARIANT_GENERIC_F4)
    for kind in TYPES:
        check(h, fmt, M, N, K, kind)
    assert sgemm.sgemm_last_variant(h)[0] == sgemm.VARIANT_GENERIC_F4


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("nt", [16, 32, 64, 128])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_every_tile_and_split(h, tile, fmt, nt, split):
    tile(nt, split)
    for M in (1, nt - 1, nt):
        for N, K in ((128, 256), (130, 2048), (300, 2500)):
            check(h, fmt, M, N, K, seed=split)
            assert sgemm.sgemm_last_variant(h) == (sgemm.VARIANT_TC_F4, min(split, max(s for s in (1, 2, 4, 8) if s <= -(-K // 256))))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 96, 127, 128, 129, 192, 255, 256, 257, 320, 511, 777, 1280, 1281])
def test_lengths(h, tile, fmt, K):
    check(h, fmt, 5, 140, K)
    tile(128, 1)
    check(h, fmt, 200, 140, K)
    tile(256, 1)
    check(h, fmt, 200, 140, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(256, 256, 256), (1, 1, 64), (129, 257, 512), (300, 300, 1500), (513, 700, 300), (1000, 1500, 777), (2100, 2300, 2000)])
def test_pairs(h, tile, fmt, M, N, K):
    tile(256, 1)
    for kind in TYPES:
        check(h, fmt, M, N, K, kind)
        assert sgemm.sgemm_last_variant(h) == (sgemm.VARIANT_TC_F4_PAIR, 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M", [1, 2, 8, 16, 17, 33, 64, 65, 128, 129, 1000])
def test_chosen(h, fmt, kind, M):
    for N, K in ((64, 200), (1000, 1024), (4100, 300)):
        check(h, fmt, M, N, K, kind, bias=M % 2 == 0, ldc=N + M % 3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [3, 150, 600])
def test_rows_on_no_boundary_are_copied(h, tile, fmt, M):
    N, K = 600, 900
    for a, b, copied in ((dict(shift=1), {}, 1), ({}, dict(pad=3), 2), (dict(shift=5, pad=0), dict(shift=8), 3)):
        check(h, fmt, M, N, K, a=a, b=b)
        assert sgemm.sgemm_last_relayout(h) == copied and sgemm.sgemm_last_launches(h) == 2
    check(h, fmt, M, N, K)
    assert sgemm.sgemm_last_relayout(h) == 0 and sgemm.sgemm_last_launches(h) == 1
    sgemm.sgemm_set_relayout(h, sgemm.RELAYOUT_OFF)
    check(h, fmt, M, N, K, a=dict(shift=1))
    assert sgemm.sgemm_last_variant(h)[0] == sgemm.VARIANT_GENERIC_F4


def test_mx_without_row_scales(h):
    for M in (4, 300):
        check(h, sgemm.FP4_MX, M, 500, 400, rows=False)


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_elements_give_the_bias(h, fmt):
    C = torch.full((3, 5), 9.0, device="cuda")
    bias, one = torch.arange(5.0, device="cuda"), torch.ones(5, device="cuda")
    sgemm.sgemm_run_fp4(h, fmt, sgemm.IN_F32, 3, 5, 0, None, 1, None, one, None, 1, None, one, bias, C, 5)
    assert torch.equal(C.cpu(), torch.arange(5.0).expand(3, 5))
    sgemm.sgemm_run_fp4(h, fmt, sgemm.IN_F32, 3, 5, 0, None, 1, None, one, None, 1, None, one, None, C, 5)
    assert (C == 0).all()


def any_rows(fmt, rows, K, gen):
    codes, scales, _ = f4.random_rows(fmt, rows, K, gen)
    span = torch.randint(100, 150, scales.shape, generator=gen) if fmt == sgemm.FP4_MX else torch.randint(0, 127, scales.shape, generator=gen)
    return codes, span.to(torch.uint8), torch.rand(rows, generator=gen) + 0.1


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(3, 200, 777), (64, 300, 2048), (300, 520, 1000), (600, 600, 4096)])
def test_scales_of_any_size(h, fmt, M, N, K):
    """Each of K terms truncated once at 2^-23 of what the sum of magnitudes can be, the
    result rounded three times more (both row scales, the bias): (K + 3) 2^-23."""
    got, want, size = product(h, fmt, M, N, K, make=any_rows, bias=False)
    assert ((got.double() - want).abs() <= (K + 3) * 2.0 ** -23 * size).all()
    # and close on the whole: K errors of 2^-23 at random, with a margin of 4
    assert float((got.double() - want).norm() / size.norm()) <= 4 * K ** 0.5 * 2.0 ** -23


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_bits_every_time(h, fmt):
    for M in (5, 100, 600):
        first, _, _ = product(h, fmt, M, 520, 3000, make=any_rows)
        for _ in range(3):
            assert torch.equal(product(h, fmt, M, 520, 3000, make=any_rows)[0], first)


def test_a_nan_scale_makes_its_products_nan(h):
    for M in (4, 300):
        def make(fmt, rows, K, gen):
            codes, scales, row = f4.random_rows(fmt, rows, K, gen)
            if rows == M:
                scales[1, 2] = 255
            return codes, scales, row
        got, want, _ = product(h, sgemm.FP4_MX, M, 140, 500, make=make, bias=False)
        assert got[1].isnan().all() and torch.equal(got[0], want[0].float()) and torch.equal(got[2:], want[2:].float())


# ---- rows to 4 bits and back ---------------------------------------------------------
def activations(M, K, gen, dtype):
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    x[:, ::7] *= 5
    if M > 2:
        x[1] = 0
        x[2, :] = torch.arange(K) % 13 - 6  # ties
    return x.to(dtype)


def special_rows(dtype, K=100):
    """Infinities, NaN, the largest and the smallest values of the type, signed zeros."""
    x = torch.ones(10, K, dtype=torch.float64)
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x[0, 40] = float("inf")
    x[1, 3] = float("nan")
    x[2] = big
    x[3] = tiny
    x[4] = tiny * torch.finfo(dtype).eps  # subnormal
    x[5] = -0.0
    x[6, 64:] = 0
    x[7, :32] *= big
    x[8, 50] = -float("inf")
    x[9, ::2] *= -tiny
    return x.to(dtype)


def quantized(h, fmt, x, shift=0, pad=None, ldx=None, off=0):
    """(codes, scales, row) of sgemm_quantize_fp4; nothing else may be written."""
    M, K = x.shape
    wide, ldx = (K + 1) // 2, ldx or K
    X = torch.full((off + M * ldx + 8,), 3.0, dtype=x.dtype)
    X[off:off + M * ldx].view(M, ldx)[:, :K] = x
    X = X.cuda()
    ld = -(-wide // 16) * 16 if pad is None else wide + pad
    Q = torch.full((shift + M * ld + 32,), 0xEE, dtype=torch.uint8, device="cuda")
    n = sgemm.sgemm_fp4_scale_bytes(fmt, M, K)
    S = torch.full((n + 64,), 0xDD, dtype=torch.uint8, device="cuda")
    row = torch.full((M + 1,), -5.0, device="cuda")
    kind = {v: k for k, v in TYPES.items()}[x.dtype]
    sgemm.sgemm_quantize_fp4(h, kind, fmt, M, K, X[off:], ldx, Q.data_ptr() + shift, ld, S, row)
    torch.cuda.synchronize()
    q, s, r = Q.cpu(), S.cpu(), row.cpu()
    body = q[shift:shift + M * ld].view(M, ld)
    assert (q[:shift] == 0xEE).all() and (q[shift + M * ld:] == 0xEE).all() and (body[:, wide:] == 0xEE).all()
    assert r[M] == -5
    index = f4.scale_index(fmt, M, K)
    words = f4.words_of(fmt, K)
    want = torch.full((n + 64,), 0xDD, dtype=torch.uint8)
    all_blocks = f4.scale_index(fmt, M, words * 4 * f4.BLOCK[fmt])
    want[all_blocks.reshape(-1)] = 0
    scales = s[index.reshape(-1)].view(index.shape)
    want[index.reshape(-1)] = scales.reshape(-1)
    assert torch.equal(s, want), "scales behind the last block must be 0, those of other rows left alone"
    if K % 2:
        assert (body[:, wide - 1] >> 4 == 0).all()
    return f4.unpack(body, K), scales, r[:M], (Q, S, row, ld)


def same_codes(got, want):
    return torch.equal(f4.code_values(got), f4.code_values(want))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES.values()))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 2), (5, 16), (4, 31), (130, 64), (7, 100), (9, 257), (300, 777), (3, 4096), (1300, 1000), (5, 17000), (700, 2050), (2, 40001)])
def test_quantize(h, fmt, dtype, M, K):
    gen = torch.Generator().manual_seed(M * K)
    x = activations(M, K, gen, dtype)
    codes, scales, m = f4.quantize(fmt, x)
    for more in (dict(), dict(shift=1, pad=1), dict(ldx=K + 3, pad=2), dict(off=1)):
        got, s, row, _ = quantized(h, fmt, x, **more)
        assert torch.equal(s, scales)
        assert same_codes(got, codes)
        assert torch.equal(row, f4.row_scales(m) if fmt == sgemm.FP4_NV else torch.ones(M))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES.values()))
def test_quantize_special_rows(h, fmt, dtype):
    x = special_rows(dtype)
    codes, scales, m = f4.quantize(fmt, x)
    got, s, row, _ = quantized(h, fmt, x)
    assert torch.equal(s, scales)
    assert same_codes(got, codes)
    want = f4.row_scales(m) if fmt == sgemm.FP4_NV else torch.ones(len(x))
    assert torch.equal(row.isnan(), want.isnan()) and torch.equal(row.nan_to_num(-1), want.nan_to_num(-1))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES.values()))
@pytest.mark.parametrize("M,K", [(1, 1), (6, 33), (130, 100), (7, 777), (40, 4096), (600, 2050)])
def test_dequantize(h, fmt, dtype, M, K):
    """One rounding to FP32 (code times scale is exact) and one to the type."""
    gen = torch.Generator().manual_seed(M + K)
    kind = {v: k for k, v in TYPES.items()}[dtype]
    for more in (dict(), dict(shift=3, pad=1), dict(pad=0)):
        A = Matrix(fmt, M, K, gen, make=any_rows, **more)
        for ldy in (K, K + 5):
            Y = torch.full((M + 1, ldy), 7.0, dtype=dtype, device="cuda")
            sgemm.sgemm_dequantize_fp4(h, kind, fmt, M, K, A.q, A.ld, A.s, A.row, Y, ldy)
            got = Y.cpu()
            assert torch.equal(got[:M, :K], A.values.float().to(dtype))
            assert (got[M] == 7).all() and (got[:M, K:] == 7).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_there_and_back_and_multiplied(h, fmt):
    """Rows quantized by the library, opened again, and multiplied: the product of what they stand for."""
    gen = torch.Generator().manual_seed(5)
    M, N, K = 70, 300, 1000
    parts = []
    for rows in (M, N):
        codes, scales, row, (Q, S, r, ld) = quantized(h, fmt, activations(rows, K, gen, torch.bfloat16))
        Y = torch.empty(rows, K, device="cuda")
        sgemm.sgemm_dequantize_fp4(h, sgemm.IN_F32, fmt, rows, K, Q, ld, S, r, Y, K)
        assert torch.equal(Y.cpu(), f4.values(fmt, codes, scales, row).float())
        parts.append((Q, ld, S, r, f4.values(fmt, codes, scales, row)))
    a, b = parts
    C = torch.empty(M, N, device="cuda")
    sgemm.sgemm_run_fp4(h, fmt, sgemm.IN_F32, M, N, K, *a[:4], *b[:4], None, C, N)
    size = a[4].abs() @ b[4].abs().T
    assert ((C.cpu().double() - a[4] @ b[4].T).abs() <= (K + 3) * 2.0 ** -23 * size + 1e-30).all()
