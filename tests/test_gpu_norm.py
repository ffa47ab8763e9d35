"""The RMS norm and its gradient on the GPU against 64-bit forms.

Tolerances, u = 2^-24 and t the type's half step (2^-24, 2^-8, 2^-11).  A sum of K
squares in FP32 errs by at most K u of itself; r takes half of that, the mean, the
addition of eps, the root and the quotient 2.5 u more: R = (K / 2 + 4) u of r, with
K the longest chain of additions (a thread's 32 elements or, in longer rows, K / 512
of them, 5 steps in a warp and 16 warps).  Y adds two products and the
rounding to the type.  The integers, codes and block scales do not depend on r: equal.
dX: the sum over K is off by C u of its magnitudes (C the chain, 3 roundings a term), what
it is multiplied with by 6 u; dweight: chain of the rows a group of threads takes, then of the
groups, all bounded by the number of rows: (M + 6) u + R of the magnitudes."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm
from tests import fp4_util as f4

pytestmark = pytest.mark.gpu

TYPES = {sgemm.IN_F32: torch.float32, sgemm.IN_BF16: torch.bfloat16, sgemm.IN_F16: torch.float16}
KINDS = {v: k for k, v in TYPES.items()}
U = 2.0 ** -24
EPS = 1e-5
SIZES = [(1, 1), (2, 3), (5, 16), (3, 33), (130, 100), (33, 257), (300, 777), (3, 4096), (1300, 1000), (5, 17000), (700, 2050), (2, 40001), (0, 64), (9, 8192)]


def chain(K):
    return max(32, -(-K // 512)) + 5 + 16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


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


def rows(M, K, gen, dtype):
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    x[:, ::7] *= 4
    if M > 3:
        x[2] = 0
    return x.to(dtype)


class Device:
    """Rows on the GPU in a buffer with elements around them that nothing may write."""

    def __init__(self, host, ld=None, off=0):
        M, K = host.shape
        self.shape, self.ld, self.off = (M, K), max(ld or K, 1), off
        full = torch.full((off + M * self.ld + 8,), 3.0, dtype=host.dtype)
        full[off:off + M * self.ld].view(M, self.ld)[:, :K] = host
        self.buf, self.before = full.cuda(), full

    @property
    def at(self):
        return self.buf[self.off:]

    def host(self, written=True):
        M, K = self.shape
        got = self.buf.cpu()
        body = got[self.off:self.off + M * self.ld].view(M, self.ld)
        out = body[:, :K].clone()
        if written:
            body[:, :K] = self.before[self.off:self.off + M * self.ld].view(M, self.ld)[:, :K]
        assert torch.equal(got.view(torch.uint8), self.before.view(torch.uint8)), "written outside of the rows"
        return out


def blank(M, K, dtype, ld=None, off=0):
    return Device(torch.full((M, K), 5.0).to(dtype), ld, off)


def case(M, K, dtype, residual, pad, off):
    gen = torch.Generator().manual_seed(M * 31 + K)
    x, w = rows(M, K, gen, dtype), (1 + 0.3 * torch.randn(1, K, generator=gen)).to(dtype)
    r = rows(M, K, gen, dtype) if residual else None
    kept = x if r is None else (x.double() + r.double()).to(torch.float32).to(dtype) if dtype == torch.float32 else (x.float() + r.float()).to(dtype)
    ld = K + pad
    return x, w, r, kept, Device(x, ld, off), Device(w, None, off), Device(r, ld, off) if residual else None


FORMS = [dict(residual=True, pad=0, off=0), dict(residual=False, pad=0, off=0), dict(residual=True, pad=1, off=1), dict(residual=True, pad=6, off=2), dict(residual=False, pad=3, off=1)]


def rstd_of(kept):
    return 1 / torch.sqrt(kept.double().square().mean(dim=1) + EPS)


@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(h, dtype, M, K):
    for form in FORMS:
        x, w, r, kept, X, W, R = case(M, K, dtype, **form)
        H, Y = blank(M, K, dtype, K + form["pad"], form["off"]), blank(M, K, dtype, K + form["pad"], form["off"])
        rstd = torch.full((M + 1,), -1.0, device="cuda")
        sgemm.sgemm_rms_norm(h, KINDS[dtype], M, K, X.at, X.ld, R and R.at, R.ld if R else 0, W.at, EPS, H.at, H.ld, Y.at, Y.ld, rstd)
        torch.cuda.synchronize()
        assert torch.equal(H.host(), kept)
        want_r, got_r = rstd_of(kept), rstd.cpu()
        assert got_r[M] == -1
        R_ERR = (chain(K) / 2 + 4) * U
        assert ((got_r[:M].double() - want_r).abs() <= R_ERR * want_r).all()
        want = kept.double() * want_r[:, None] * w.double()
        t, tiny = half_step(dtype), float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
        assert ((Y.host().double() - want).abs() <= ((1 + R_ERR + 3 * U) * (1 + t) - 1) * want.abs() + tiny).all()


@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_to_8_bits(h, dtype, M, K):
    for form in FORMS:
        x, w, r, kept, X, W, R = case(M, K, dtype, **form)
        H = blank(M, K, dtype) if form["residual"] else None
        Q = Device(torch.zeros(M, K, dtype=torch.int8), K + form["pad"], form["off"])
        scale = torch.full((M + 1,), -1.0, device="cuda")
        sgemm.sgemm_rms_norm_int8(h, KINDS[dtype], M, K, X.at, X.ld, R and R.at, R.ld if R else 0, W.at, EPS, H and H.at, K, Q.at, Q.ld, scale)
        torch.cuda.synchronize()
        if H:
            assert torch.equal(H.host(), kept)
        v = kept.float() * w.float()
        m = v.abs().amax(dim=1)
        inv = torch.where(m > 0, torch.tensor(127.0) / m, torch.zeros_like(m))
        assert torch.equal(Q.host(), torch.round(v * inv[:, None]).to(torch.int8))
        want = m.double() * rstd_of(kept) / 127
        assert ((scale.cpu()[:M].double() - want).abs() <= (chain(K) / 2 + 6) * U * want).all()


@pytest.mark.parametrize("fmt", [sgemm.FP4_MX, sgemm.FP4_NV])
@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("M,K", [s for s in SIZES if s[0]])
def test_norm_to_4_bits(h, fmt, dtype, M, K):
    for form in FORMS:
        x, w, r, kept, X, W, R = case(M, K, dtype, **form)
        H = blank(M, K, dtype) if form["residual"] else None
        wide = (K + 1) // 2
        Q = Device(torch.zeros(M, wide, dtype=torch.uint8), wide + form["pad"], form["off"])
        S = torch.zeros(sgemm.sgemm_fp4_scale_bytes(fmt, M, K), dtype=torch.uint8, device="cuda")
        row = torch.full((M + 1,), -1.0, device="cuda")
        sgemm.sgemm_rms_norm_fp4(h, KINDS[dtype], fmt, M, K, X.at, X.ld, R and R.at, R.ld if R else 0, W.at, EPS, H and H.at, K, Q.at, Q.ld, S, row)
        torch.cuda.synchronize()
        codes, scales, m = f4.quantize(fmt, kept.float() * w.float())
        got = f4.unpack(Q.host(), K)
        assert torch.equal(f4.code_values(got), f4.code_values(codes))
        assert torch.equal(S.cpu(), f4.tiled(fmt, scales, K))
        want = rstd_of(kept) if fmt == sgemm.FP4_MX else m.double() / 2688 * rstd_of(kept)
        assert ((row.cpu()[:M].double() - want).abs() <= (chain(K) / 2 + 6) * U * want).all()


@pytest.mark.parametrize("dtype", list(KINDS))
def test_rows_with_infinities_and_nan(h, dtype):
    K = 200
    x = torch.ones(4, K)
    x[1, 7], x[2, 199] = float("inf"), float("nan")
    X, W = Device(x.to(dtype)), Device(torch.ones(1, K).to(dtype))
    Q, scale = Device(torch.ones(4, K, dtype=torch.int8)), torch.zeros(4, device="cuda")
    sgemm.sgemm_rms_norm_int8(h, KINDS[dtype], 4, K, X.at, K, None, 0, W.at, EPS, None, 0, Q.at, K, scale)
    assert scale.cpu().isnan().tolist() == [False, True, True, False]
    assert (Q.host()[1:3] == 0).all() and (Q.host()[::3] == 127).all()
    Y = blank(4, K, dtype)
    sgemm.sgemm_rms_norm(h, KINDS[dtype], 4, K, X.at, K, None, 0, W.at, EPS, None, 0, Y.at, K, None)
    y = Y.host().float()
    assert y[2].isnan().all() and y[1, 7].isnan() and (y[1, :7] == 0).all() and torch.equal(y[0], y[3])
    row = torch.zeros(4, device="cuda")
    for fmt in (sgemm.FP4_MX, sgemm.FP4_NV):
        S = torch.zeros(sgemm.sgemm_fp4_scale_bytes(fmt, 4, K), dtype=torch.uint8, device="cuda")
        Q = Device(torch.ones(4, K // 2, dtype=torch.uint8))
        sgemm.sgemm_rms_norm_fp4(h, KINDS[dtype], fmt, 4, K, X.at, K, None, 0, W.at, EPS, None, 0, Q.at, K // 2, S, row)
        s = S.cpu()[f4.scale_index(fmt, 4, K)]
        if fmt == sgemm.FP4_NV:
            assert row.cpu().isnan().tolist() == [False, True, True, False] and (s[1:3] == 0).all()
        else:
            assert s[1, 0] == 255 and s[2, 6] == 255 and (s[0] != 255).all()


@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("K", [64, 300, 20000])
def test_sum_in_place_of_either_row(h, dtype, K):
    for which in (0, 1):
        x, w, r, kept, X, W, R = case(37, K, dtype, True, 0, 0)
        into = (X, R)[which]
        Q, scale = Device(torch.zeros(37, K, dtype=torch.int8)), torch.zeros(37, device="cuda")
        sgemm.sgemm_rms_norm_int8(h, KINDS[dtype], 37, K, X.at, K, R.at, K, W.at, EPS, into.at, K, Q.at, K, scale)
        torch.cuda.synchronize()
        assert torch.equal(into.host(), kept)
        v = kept.float() * w.float()
        m = v.abs().amax(dim=1)
        assert torch.equal(Q.host(), torch.round(v * torch.where(m > 0, torch.tensor(127.0) / m, torch.zeros_like(m))[:, None]).to(torch.int8))


def grad_reference(dy, dh, kept, w, r):
    dy, x, w = dy.double(), kept.double(), w.double()
    g, r, K = dy * w, r.double()[:, None], x.shape[1]
    inner, size = (g * x).sum(1, keepdim=True), (g * x).abs().sum(1, keepdim=True)
    dx = r * g - x * r ** 3 / K * inner
    bound = (r * g).abs() + x.abs() * r ** 3 / K * size
    if dh is not None:
        dx, bound = dx + dh.double(), bound + dh.double().abs()
    return dx, bound, (dy * x * r).sum(0), (dy * x * r).abs().sum(0)


@pytest.mark.parametrize("dtype", list(KINDS))
@pytest.mark.parametrize("M,K", [s for s in SIZES if s[0]] + [(2000, 130), (700, 4096), (400, 16384), (3000, 16), (1300, 2056), (2000, 8192), (1500, 5000)])
def test_gradient(h, dtype, M, K):
    gen = torch.Generator().manual_seed(M + K)
    for form in (FORMS[0], FORMS[1], FORMS[2]):
        x, w, r, kept, X, W, R = case(M, K, dtype, False, form["pad"], form["off"])
        dy, dh = rows(M, K, gen, dtype), rows(M, K, gen, dtype) if form["residual"] else None
        rstd = rstd_of(kept).float()
        dY, dH, dX = Device(dy, K + form["pad"], form["off"]), Device(dh, K + form["pad"], form["off"]) if dh is not None else None, blank(M, K, dtype, K + form["pad"], form["off"])
        dw, r_dev = torch.full((K + 1,), 9.0, device="cuda"), rstd.cuda()
        call = lambda: sgemm.sgemm_rms_norm_grad(h, KINDS[dtype], M, K, dY.at, dY.ld, dH and dH.at, dH.ld if dH else 0, X.at, X.ld, W.at, r_dev, dX.at, dX.ld, dw)  # noqa: E731
        call()
        torch.cuda.synchronize()
        want, bound, want_w, bound_w = grad_reference(dy, dh, kept, w, rstd)
        t = half_step(dtype)
        tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
        got, got_w = dX.host(), dw.cpu()
        assert got_w[K] == 9
        assert ((got.double() - want).abs() <= (chain(K) + 10) * U * bound + t * (want.abs() + (chain(K) + 10) * U * bound) + tiny).all()
        assert ((got_w[:K].double() - want_w).abs() <= (M + 6) * U * bound_w).all()
        call()
        assert torch.equal(dX.host(), got) and torch.equal(dw.cpu(), got_w), "the same bits every time"


def test_gradient_in_place_and_without_rows(h):
    gen = torch.Generator().manual_seed(8)
    x, w, _, kept, X, W, _ = case(40, 500, torch.float32, False, 0, 0)
    dy, dh = rows(40, 500, gen, torch.float32), rows(40, 500, gen, torch.float32)
    r = rstd_of(kept).float()
    dY, A, B = Device(dy), Device(dh), blank(40, 500, torch.float32)
    dw = torch.ones(500, device="cuda")
    sgemm.sgemm_rms_norm_grad(h, 0, 40, 500, dY.at, 500, A.at, 500, X.at, 500, W.at, r.cuda(), B.at, 500, dw)
    sgemm.sgemm_rms_norm_grad(h, 0, 40, 500, dY.at, 500, A.at, 500, X.at, 500, W.at, r.cuda(), A.at, 500, dw)
    assert torch.equal(A.host(), B.host())
    sgemm.sgemm_rms_norm_grad(h, 0, 0, 500, None, 500, None, 0, None, 500, None, None, None, 500, dw)
    assert (dw == 0).all()


def test_gradient_against_differences(h):
    """d loss / d x and w of loss = <Y, c> + <H, d> by central differences of the 64-bit form: their
    error is of the order of step^2, 1e-6 of values around 1."""
    gen = torch.Generator().manual_seed(3)
    M, K = 3, 24
    x, w, c, d = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((M, K), (K,), (M, K), (M, K)))

    def loss(x, w):
        return float(((x * rstd_of(x)[:, None] * w) * c + x * d).sum())
    step = 1e-4
    num_x, num_w = torch.zeros_like(x), torch.zeros_like(w)
    for t, num in ((x, num_x), (w, num_w)):
        for i in range(t.numel()):
            for sign in (1, -1):
                t.view(-1)[i] += sign * step
                num.view(-1)[i] += sign * loss(x, w) / (2 * step)
                t.view(-1)[i] -= sign * step
    X, W, dY, dH, dX = Device(x.float()), Device(w.float()[None]), Device(c.float()), Device(d.float()), blank(M, K, torch.float32)
    Y, rstd, dw = blank(M, K, torch.float32), torch.zeros(M, device="cuda"), torch.zeros(K, device="cuda")
    sgemm.sgemm_rms_norm(h, 0, M, K, X.at, K, None, 0, W.at, EPS, None, 0, Y.at, K, rstd)
    sgemm.sgemm_rms_norm_grad(h, 0, M, K, dY.at, K, dH.at, K, X.at, K, W.at, rstd, dX.at, K, dw)
    scale = float(num_x.abs().max())
    assert float((dX.host().double() - num_x).abs().max()) <= 1e-5 * scale
    assert float((dw.cpu().double() - num_w).abs().max()) <= 1e-5 * float(num_w.abs().max())
