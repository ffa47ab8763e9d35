"""GPU parity of the int8 products (sgemm_run_int8, sgemm_run_int8_experts)
and of sgemm_quantize_rows against plain 64-bit forms.

Tolerance of a product: the integer sum is exact and the kernels compute
fl(fma(fl(fl(sum) * sb), sa, bias)) with three FP32 roundings before the one to
the output type, so |C - exact| <= 3.1 * 2^-24 * |sum sa sb| + 2^-24 * |exact|
+ u * |exact| (1 + 2^-20) + tiny, u = 0, 2^-8, 2^-11 (the unit roundoff of 8 and
11 significant bits, 2^-p: half the spacing 2^(1-p) of the values just above 1;
the FP32 rounding is the 2^-24 term) and tiny = 2^-25 for FP16's subnormals.  With scales of 1 and no bias, FP32 results are the integer
rounded to FP32 and must be equal bit for bit."""
import numpy as np
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm

pytestmark = pytest.mark.gpu

V = sgemm
TYPES = {"f32": (V.IN_F32, torch.float32, 0.0), "bf16": (V.IN_BF16, torch.bfloat16, 2.0 ** -8),
         "f16": (V.IN_F16, torch.float16, 2.0 ** -11)}
FILL = 77.0  # what C holds before a call


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    h = sgemm.sgemm_create()
    yield h
    assert sgemm.sgemm_get_device_status(h) == V.OK
    sgemm.sgemm_destroy(h)


@pytest.fixture
def pinned(handle):
    def pin(v):
        sgemm.sgemm_set_variant(handle, v)
    yield pin
    sgemm.sgemm_set_variant(handle, V.VARIANT_AUTO)
    sgemm.sgemm_set_relayout(handle, V.RELAYOUT_AUTO)


def integers(g, *shape, kind="random"):
    if kind == "low":
        return torch.full(shape, -128, dtype=torch.int8)
    if kind == "high":
        return torch.full(shape, 127, dtype=torch.int8)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int16).to(torch.int8)


def strided(x, pad, offset=0, fill=85):
    """x on the GPU with rows `pad` longer, starting `offset` elements into its buffer; the rest holds `fill`."""
    rows, cols = x.shape
    flat = torch.full((offset + rows * (cols + pad) + 64,), fill, dtype=x.dtype, device="cuda")
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view, flat


def addr(view, flat, offset):
    return flat.data_ptr() + offset * flat.element_size()


class Problem:
    def __init__(self, M, N, K, dtype="f32", trans_b=1, bias=False, pads=(0, 0, 0), offsets=(0, 0, 0), kind="random",
                 unit=False, seed=0):
        g = torch.Generator().manual_seed(seed * 7919 + M * 31 + N * 17 + K)
        self.M, self.N, self.K, self.trans_b = M, N, K, trans_b
        self.kind, self.type, self.u = TYPES[dtype]
        self.a = integers(g, M, K, kind=kind)
        self.b = integers(g, N, K, kind=kind)          # as N x K; stored as trans_b says
        self.sa = torch.ones(M) if unit else torch.rand(M, generator=g) + 0.5
        self.sb = torch.ones(N) if unit else (torch.rand(N, generator=g) + 0.5) / 512
        self.bias = torch.randn(N, generator=g) if bias else None
        self.A, self.Af = strided(self.a, pads[0], offsets[0])
        self.B, self.Bf = strided(self.b if trans_b else self.b.t().contiguous(), pads[1], offsets[1])
        self.C, self.Cf = strided(torch.full((M, N), FILL, dtype=self.type), pads[2], offsets[2], fill=FILL)
        self.pads, self.offsets = pads, offsets
        self.SA, self.SB = self.sa.cuda(), self.sb.cuda()
        self.Bias = None if self.bias is None else self.bias.cuda()

    def run(self, h, stream=None):
        sgemm.sgemm_run_int8(h, self.trans_b, self.kind, self.M, self.N, self.K, addr(self.A, self.Af, self.offsets[0]),
                             max(self.K + self.pads[0], 1), self.SA, addr(self.B, self.Bf, self.offsets[1]),
                             max((self.K if self.trans_b else self.N) + self.pads[1], 1), self.SB, self.Bias,
                             addr(self.C, self.Cf, self.offsets[2]), self.N + self.pads[2], stream)
        torch.cuda.synchronize()
        return self.C.cpu()

    def exact(self):
        sums = self.a.double().cuda() @ self.b.double().cuda().t()   # integers below 2^53: exact
        prod = sums.cpu() * self.sb.double() * self.sa.double()[:, None]
        return prod, prod + (0 if self.bias is None else self.bias.double())

    def check(self, got):
        prod, want = self.exact()
        tol = 3.1 * 2.0 ** -24 * prod.abs() + (2.0 ** -24 + self.u * (1 + 2.0 ** -20)) * want.abs()
        if self.type == torch.float16:
            tol = tol + 2.0 ** -25
            keep = want.abs() < 65000
        else:
            keep = torch.ones_like(want, dtype=torch.bool)
        bad = ((got.double() - want).abs() > tol) & keep
        if bad.any():
            i, j = (int(x) for x in bad.nonzero()[0])
            raise AssertionError(f"{int(bad.sum())} of {bad.numel()} beyond the tolerance; C[{i}][{j}] = "
                                 f"{float(got[i, j])!r}, exact {float(want[i, j])!r}")
        # nothing outside C's window was written
        full = self.Cf.clone()
        o = self.offsets[2]
        full[o:o + self.M * (self.N + self.pads[2])].view(self.M, -1)[:, :self.N] = FILL
        assert bool((full == FILL).all()), "cells outside C were written"


# every token tile and both sides of its end, channels and k on both sides of their tiles
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 300, 1000), (2, 129, 127), (15, 127, 129), (16, 256, 64), (17, 130, 1024),
          (31, 64, 1025), (32, 128, 2049), (33, 500, 96), (63, 257, 300), (64, 384, 512), (65, 128, 640),
          (127, 200, 1023), (128, 129, 1152), (129, 1000, 33), (300, 300, 300), (257, 640, 4097), (1000, 96, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_parity(handle, M, N, K, dtype):
    p = Problem(M, N, K, dtype, bias=(M + N) % 2 == 0, seed=1)
    p.check(p.run(handle))


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (17, 130, 777), (129, 257, 1025), (70, 64, 40)])
@pytest.mark.parametrize("trans_b", [0, 1])
@pytest.mark.parametrize("pads,offsets", [((0, 0, 0), (0, 0, 0)), ((3, 0, 5), (0, 0, 0)), ((16, 16, 4), (16, 16, 4)),
                                          ((1, 7, 1), (3, 5, 1)), ((0, 0, 0), (1, 1, 1))])
def test_layouts_strides_and_alignment(handle, pinned, M, N, K, trans_b, pads, offsets):
    pinned(V.VARIANT_TC_I8)
    p = Problem(M, N, K, "bf16", trans_b=trans_b, bias=True, pads=pads, offsets=offsets, seed=2)
    p.check(p.run(handle))
    in_place = trans_b and (K + pads[1]) % 16 == 0 and offsets[1] % 16 == 0
    assert sgemm.sgemm_last_relayout(handle) == (0 if in_place else 2)
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_TC_I8


@pytest.mark.parametrize("kind", ["low", "high", "random"])
@pytest.mark.parametrize("M,N,K", [(5, 130, 1024), (40, 128, 1023), (20, 64, 1152), (130, 140, 9000)])
def test_sums_are_exact_integers(handle, kind, M, N, K):
    """-128 * -128 * 1024 = 2^24 is the largest sum an FP32 accumulator is given; beyond, int32 takes over."""
    p = Problem(M, N, K, "f32", kind=kind, unit=True, seed=3)
    if kind == "high":
        p.a[:, ::3] = 125          # odd sums near 2^24
        p.A.copy_(p.a)
    got = p.run(handle)
    want = (p.a.double().cuda() @ p.b.double().cuda().t()).cpu().float()
    assert torch.equal(got, want)


@pytest.mark.parametrize("variant", [V.VARIANT_GENERIC_I8, V.VARIANT_GENERIC])
@pytest.mark.parametrize("trans_b", [0, 1])
def test_generic_variant_gives_the_same_bits(handle, pinned, variant, trans_b):
    for M, N, K in [(3, 70, 65), (100, 129, 1500)]:
        p = Problem(M, N, K, "f16", trans_b=trans_b, bias=True, pads=(1, 2, 3), seed=4)
        pinned(V.VARIANT_TC_I8)
        first = p.run(handle)
        assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_TC_I8
        pinned(variant)
        assert torch.equal(p.run(handle).view(torch.int16), first.view(torch.int16))
        assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_GENERIC_I8
        p.check(first)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 15), (130, 16), (33, 17), (129, 496), (64, 511), (70, 1000), (3, 5000), (2000, 300)])
@pytest.mark.parametrize("pads,offsets", [((0, 0, 0), (0, 0, 0)), ((16, 32, 2), (16, 16, 2)), ((1, 7, 1), (3, 5, 1)),
                                          ((0, 4, 0), (2, 8, 0)), ((5, 1, 0), (0, 15, 3))])
def test_few_tokens(handle, pinned, M, N, K, pads, offsets):
    """The kernel for up to 8 tokens against the exact form and, bit for bit, the generic one."""
    p = Problem(M, N, K, ["f32", "bf16", "f16"][M % 3], bias=N % 2 == 0, pads=pads, offsets=offsets, seed=10)
    pinned(V.VARIANT_FEW_I8)
    first = p.run(handle)
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_FEW_I8 and sgemm.sgemm_last_launches(handle) == 1
    p.check(first)
    pinned(V.VARIANT_GENERIC_I8)
    assert torch.equal(p.run(handle), first)


def test_few_tokens_at_the_extremes(handle, pinned):
    """Its sums are the integers at -128 * -128 too, and calls beyond its reach run elsewhere."""
    pinned(V.VARIANT_FEW_I8)
    p = Problem(3, 40, 16000, "f32", kind="low", unit=True, seed=11)
    assert torch.equal(p.run(handle), (p.a.double() @ p.b.double().t()).float())
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_FEW_I8
    for M, K, trans_b in [(9, 64, 1), (3, 16400, 1), (2, 64, 0)]:   # rows, shared memory, layout
        q = Problem(M, 40, K, "f32", trans_b=trans_b, seed=12)
        q.check(q.run(handle))
        assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_TC_I8


def test_relayout_off_runs_the_generic_kernel(handle, pinned):
    p = Problem(20, 50, 60, "f32", trans_b=0, seed=5)
    sgemm.sgemm_set_relayout(handle, V.RELAYOUT_OFF)
    p.check(p.run(handle))
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_GENERIC_I8
    sgemm.sgemm_set_relayout(handle, V.RELAYOUT_AUTO)


@pytest.mark.parametrize("N", [72, 1024])
def test_longest_k(handle, N):
    """K at its limit.  With the wider B the tokens are expanded to FP16 (256 KiB a
    row), more than the workspace holds at once: several passes."""
    p = Problem(2100, N, 131071, "f32", unit=True, seed=6)
    got = p.run(handle)
    assert torch.equal(got, (p.a.double().cuda() @ p.b.double().cuda().t()).cpu().float())
    assert sgemm.sgemm_last_launches(handle) > 3 or N == 72


def test_no_products(handle):
    p = Problem(7, 9, 0, "bf16", bias=True, seed=7)
    p.check(p.run(handle))
    z = torch.zeros(4, device="cuda")
    sgemm.sgemm_run_int8(handle, 1, V.IN_F32, 0, 5, 5, None, 5, None, None, 5, None, None, None, 5)
    sgemm.sgemm_run_int8(handle, 1, V.IN_F32, 5, 0, 5, None, 5, None, None, 5, None, None, None, 1)
    assert sgemm.sgemm_last_launches(handle) == 0
    assert bool((z == 0).all())


def test_special_scales(handle):
    """A NaN or infinite scale reaches its own row or column only."""
    p = Problem(20, 140, 256, "f32", seed=8)
    p.SA[3] = float("nan")
    p.SB[130] = float("inf")
    got = p.run(handle)
    assert bool(got[3].isnan().all())
    rest = got[torch.arange(20) != 3][:, torch.arange(140) != 130]
    assert bool(rest.isfinite().all())


def test_another_stream_and_a_graph(handle):
    p = Problem(48, 256, 512, "f16", seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.check(p.run(handle, s))
    p.C.fill_(FILL)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgemm.sgemm_run_int8(handle, 1, p.kind, 48, 256, 512, p.A, 512, p.SA, p.B, 512, p.SB, None, p.C, 256)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    p.check(p.C.cpu())


def test_refusals(handle):
    t = torch.zeros(4096, device="cuda")
    i8 = torch.zeros(4096, dtype=torch.int8, device="cuda")
    j8 = torch.zeros(4096, dtype=torch.int8, device="cuda")

    def status(**k):
        d = dict(transB=1, out_type=V.IN_F32, M=4, N=8, K=16, A=i8, lda=16, scaleA=t.data_ptr() + 4096, B=j8, ldb=16,
                 scaleB=t.data_ptr() + 8192, bias=None, C=t, ldc=8)
        d.update(k)
        try:
            sgemm.sgemm_run_int8(handle, **d)
        except sgemm.SgemmError as e:
            return e.status
        return V.OK

    assert status() == V.OK
    for bad in (dict(transB=2), dict(out_type=3), dict(M=-1), dict(N=-1), dict(K=-1), dict(K=131072, lda=131072, ldb=131072),
                dict(lda=15), dict(ldb=15), dict(ldc=7), dict(C=t.data_ptr() + 2), dict(scaleA=t.data_ptr() + 4097)):
        assert status(**bad) == V.ERR_INVALID_VALUE, bad
    for bad in (dict(A=None), dict(B=None), dict(C=None), dict(scaleA=None), dict(scaleB=None)):
        assert status(**bad) == V.ERR_NULL, bad
    assert status(C=t, scaleA=t) == V.ERR_ALIAS
    assert status(C=i8) == V.ERR_ALIAS
    torch.cuda.synchronize()


# ---------------------------------------------------------------- experts
class Experts:
    def __init__(self, counts, N, K, dtype="f32", trans_b=1, bias=False, before=0, after=0, seed=0, shared=False, pad=0):
        g = torch.Generator().manual_seed(seed + 1000 * len(counts) + N)
        self.counts, self.N, self.K, self.E, self.trans_b = counts, N, K, len(counts), trans_b
        self.before, self.R = before, before + sum(counts) + after
        self.kind, self.type, self.u = TYPES[dtype]
        self.a = integers(g, self.R, K)
        self.b = integers(g, 1 if shared else self.E, N, K)
        self.sa = torch.rand(self.R, generator=g) + 0.5
        self.sb = (torch.rand(self.E, N, generator=g) + 0.5) / 512
        self.bias = torch.randn(self.E, N, generator=g) if bias else None
        self.offsets = torch.tensor([before + sum(counts[:i]) for i in range(self.E + 1)], dtype=torch.int32)
        stored = self.b if trans_b else self.b.transpose(1, 2)
        self.Bf = torch.nn.functional.pad(stored, (0, pad)).contiguous().cuda()
        self.ldb = self.Bf.shape[2]
        self.strideB = 0 if shared else self.Bf.shape[1] * self.ldb
        self.dev = [x.cuda() if x is not None else None for x in (self.a, self.sa, self.sb, self.bias, self.offsets)]
        self.C = torch.full((self.R + 1, N), FILL, dtype=self.type, device="cuda")

    def run(self, h, offsets=None):
        a, sa, sb, bias, off = self.dev
        sgemm.sgemm_run_int8_experts(h, self.trans_b, self.kind, self.E, self.R, self.N, self.K,
                                     off if offsets is None else offsets, a, self.K, sa, self.Bf, self.ldb,
                                     self.strideB, sb, bias, self.C, self.N)
        torch.cuda.synchronize()
        return self.C.cpu()

    def check(self, got):
        want = torch.full((self.R + 1, self.N), FILL, dtype=torch.float64)
        tol = torch.zeros_like(want)
        for e in range(self.E):
            r0, r1 = int(self.offsets[e]), int(self.offsets[e + 1])
            w = self.b[e if self.b.shape[0] > 1 else 0]
            prod = (self.a[r0:r1].double() @ w.double().t()) * self.sb[e].double() * self.sa[r0:r1].double()[:, None]
            want[r0:r1] = prod + (0 if self.bias is None else self.bias[e].double())
            tol[r0:r1] = 3.1 * 2.0 ** -24 * prod.abs() + (2.0 ** -24 + self.u * (1 + 2.0 ** -20)) * want[r0:r1].abs()
        if self.type == torch.float16:
            tol += 2.0 ** -25
        bad = (got.double() - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("counts", [[5], [0, 3, 0, 1], [16, 17, 15, 0, 1], [130, 0, 64, 129], [0] * 40 + [2] + [1] * 25,
                                    [300, 1, 128]])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_experts_parity(handle, counts, dtype):
    p = Experts(counts, 200, 160, dtype, bias=len(counts) % 2 == 0, seed=1)
    p.check(p.run(handle))


@pytest.mark.parametrize("K", [16, 1024, 1040, 3000])
def test_experts_rows_without_an_expert_stay(handle, K):
    p = Experts([7, 0, 20], 130, K, "bf16", before=3, after=9, seed=2)
    p.check(p.run(handle))


@pytest.mark.parametrize("trans_b,pad,shared", [(0, 0, False), (0, 5, False), (1, 1, False), (1, 0, True), (0, 0, True)])
def test_experts_layouts(handle, trans_b, pad, shared):
    p = Experts([7, 33, 0, 12], 150, 272, "f32", trans_b=trans_b, pad=pad, shared=shared, bias=True, seed=3)
    p.check(p.run(handle))
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_TC_I8


def test_experts_generic_gives_the_same_bits(handle, pinned):
    p = Experts([7, 33, 0, 12], 150, 272, "f32", bias=True, before=2, after=2, seed=4)
    first = p.run(handle)
    pinned(V.VARIANT_GENERIC_I8)
    p.C.fill_(FILL)
    assert torch.equal(p.run(handle), first)
    p.check(first)


def test_experts_no_rows_at_all(handle):
    p = Experts([0, 0, 0], 64, 64, "f32", after=5, seed=5)
    p.check(p.run(handle))


@pytest.mark.parametrize("bad", [[0, 50, 20, 30], [-5, 10, 999, 40], [40, 30, 20, 10], [999, 999, 999, 999]])
@pytest.mark.parametrize("variant", [V.VARIANT_AUTO, V.VARIANT_GENERIC_I8])
def test_experts_offsets_out_of_order_stay_in_bounds(handle, pinned, bad, variant):
    p = Experts([10, 20, 10], 64, 64, "f32", seed=6)
    pinned(variant)
    got = p.run(handle, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert bool((got[p.R] == FILL).all())
    assert sgemm.sgemm_get_device_status(handle) == V.OK


def test_experts_refusals(handle):
    p = Experts([4], 16, 16, "f32", seed=7)
    a, sa, sb, _, off = p.dev

    def status(**k):
        d = dict(transB=1, out_type=V.IN_F32, experts=1, rows=4, N=16, K=16, offsets=off, A=a, lda=16, scaleA=sa,
                 B=p.Bf, ldb=16, strideB=256, scaleB=sb, bias=None, C=p.C, ldc=16)
        d.update(k)
        try:
            sgemm.sgemm_run_int8_experts(handle, **d)
        except sgemm.SgemmError as e:
            return e.status
        return V.OK

    assert status() == V.OK
    for bad in (dict(experts=0), dict(experts=1025), dict(strideB=-1), dict(rows=-1), dict(ldc=15)):
        assert status(**bad) == V.ERR_INVALID_VALUE, bad
    assert status(offsets=None) == V.ERR_NULL
    assert status(C=p.dev[0]) == V.ERR_ALIAS
    torch.cuda.synchronize()


# -------------------------------------------------------------- quantization
def plain_quantize(x):
    """In 64 bits where it can be: the FP32 roundings that the contract states are applied one by one."""
    x = x.float().numpy().astype(np.float32)
    m = np.abs(x).max(axis=1, initial=0).astype(np.float32)
    finite = np.isfinite(x).all(axis=1)
    small = ~(m >= np.float32(127 * 2.0 ** -126))
    with np.errstate(all="ignore"):
        inv = (np.float32(127) / m).astype(np.float32)
        prod = (x * inv[:, None]).astype(np.float32)
        q = np.rint(prod.astype(np.float64))
    q[small | ~finite] = 0
    scale = (m / np.float32(127)).astype(np.float32)
    scale[small] = 0
    scale[~finite] = np.nan
    return q.astype(np.int8), scale


QUANT_SHAPES = [(1, 1), (3, 7), (1, 16), (5, 255), (2, 256), (700, 64), (3, 1025), (2, 4096), (650, 2000), (3, 8193),
                (2, 40000), (1, 16385)]


@pytest.mark.parametrize("M,K", QUANT_SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
def test_quantize(handle, M, K, dtype, pad, offset):
    g = torch.Generator().manual_seed(M * 131 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))).to(TYPES[dtype][1])
    if M > 2:
        x[1] = 0
    X, Xf = strided(x, pad, offset, fill=1.0e4)
    Q, Qf = strided(torch.full((M, K), 99, dtype=torch.int8), pad, offset, fill=99)
    scale = torch.full((M + 1,), -1.0, device="cuda")
    sgemm.sgemm_quantize_rows(handle, TYPES[dtype][0], M, K, addr(X, Xf, offset), K + pad, addr(Q, Qf, offset), K + pad,
                              scale)
    torch.cuda.synchronize()
    want_q, want_s = plain_quantize(x)
    assert np.array_equal(scale[:M].cpu().numpy(), want_s) and float(scale[M]) == -1.0
    assert np.array_equal(Q.cpu().numpy(), want_q)
    Q.fill_(99)
    assert bool((Qf == 99).all())


def test_quantize_ties_and_special_rows(handle):
    x = torch.zeros(9, 40)
    x[0, :5] = torch.tensor([127.0, 0.5, 1.5, -0.5, -2.5])      # ties go to the even integer
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    x[3, 3] = -float("inf")
    x[4, 3] = 1e-40                                             # below the smallest row maximum
    x[5, 3] = 127 * 2.0 ** -126
    x[6, 3] = 3.4028234e38
    x[7] = torch.linspace(-1, 1, 40)
    x[8, 0] = -0.0
    X, q, s = x.cuda(), torch.zeros(9, 40, dtype=torch.int8, device="cuda"), torch.zeros(9, device="cuda")
    sgemm.sgemm_quantize_rows(handle, V.IN_F32, 9, 40, X, 40, q, 40, s)
    torch.cuda.synchronize()
    want_q, want_s = plain_quantize(x)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    assert q[0, :5].tolist() == [127, 0, 2, 0, -2]


def test_quantize_empty_and_refusals(handle):
    s = torch.full((4,), 5.0, device="cuda")
    x = torch.zeros(256, device="cuda")
    q = torch.zeros(256, dtype=torch.int8, device="cuda")
    sgemm.sgemm_quantize_rows(handle, V.IN_F32, 0, 8, None, 8, None, 8, None)
    sgemm.sgemm_quantize_rows(handle, V.IN_F32, 4, 0, None, 1, None, 1, s)
    torch.cuda.synchronize()
    assert s.tolist() == [0, 0, 0, 0]

    def status(**k):
        d = dict(in_type=V.IN_F32, M=4, K=8, X=x, ldx=8, Q=q, ldq=8, scale=s)
        d.update(k)
        try:
            sgemm.sgemm_quantize_rows(handle, **d)
        except sgemm.SgemmError as e:
            return e.status
        return V.OK

    assert status() == V.OK
    for bad in (dict(in_type=3), dict(in_type=-1), dict(M=-1), dict(K=-1), dict(ldx=7), dict(ldq=7),
                dict(X=x.data_ptr() + 2), dict(scale=s.data_ptr() + 1)):
        assert status(**bad) == V.ERR_INVALID_VALUE, bad
    for bad in (dict(X=None), dict(Q=None), dict(scale=None)):
        assert status(**bad) == V.ERR_NULL, bad
    assert status(Q=x) == V.ERR_ALIAS
    assert status(scale=x) == V.ERR_ALIAS
    torch.cuda.synchronize()
