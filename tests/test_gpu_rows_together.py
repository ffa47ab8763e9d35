"""The norm, 4-bit and expert-layer calls as they are used together: one behind the
other in the same buffers, in CUDA graphs, on streams that are not the current one, on
buffers past 2^31 elements, through the tensor methods and the example."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from examples import expert_layer as ex
from tests import fp4_util as f4
from tests.test_gpu_tensor_streams import DELAY, tensors

pytestmark = pytest.mark.gpu

V = sgemm
FORMATS = [V.FP4_MX, V.FP4_NV]
EPS = 1e-5


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    with sgemm.Sgemm() as handle:
        yield handle
        torch.cuda.synchronize()
        assert handle.device_status() == sgemm.OK


class Step:
    """One layer's calls on buffers of its own: norm with the residual to 4 bits, weights quantized
    anew, the product, its result's norm to 8 bits, an int8 product, then a whole expert layer on the
    product's first rows."""

    def __init__(self, fmt, M, N, K, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        bf, u8, f32, i8 = torch.bfloat16, torch.uint8, torch.float32, torch.int8
        self.fmt, self.M, self.N, self.K, self.wide = fmt, M, N, K, -(-K // 32) * 16
        self.x = [randn(M, K).bfloat16() for _ in range(3)]
        self.w = [randn(N, K).bfloat16() for _ in range(2)]
        self.residual, self.norm = new(M, K, dtype=bf), (1 + randn(K) / 5).bfloat16()
        self.qa, self.qb = new(M, self.wide, dtype=u8), new(N, self.wide, dtype=u8)
        self.sa, self.sb = (new(V.sgemm_fp4_scale_bytes(fmt, r, K), dtype=u8) for r in (M, N))
        self.ra, self.rb = new(M, dtype=f32), new(N, dtype=f32)
        self.y, self.norm2 = new(M, N, dtype=bf), (1 + randn(N) / 5).bfloat16()
        self.q8, self.s8, self.z = new(M, N, dtype=i8), new(M, dtype=f32), new(M, 96, dtype=bf)
        self.b8, self.sb8 = torch.randint(-127, 128, (96, N), generator=gen, device="cuda", dtype=i8), torch.rand(96, generator=gen, device="cuda")
        self.T, self.E, self.F = min(M, 12), 4, 64
        self.ids = [torch.randint(-1, self.E, (self.T, 2), generator=gen, device="cuda", dtype=torch.int32) for _ in range(3)]
        self.route, self.cw = new(self.T, 2, dtype=torch.int32), torch.rand(self.T, 2, generator=gen, device="cuda")
        self.up, self.us = torch.randint(-127, 128, (self.E, 2 * self.F, N), generator=gen, device="cuda", dtype=i8), torch.rand(self.E, 2 * self.F, generator=gen, device="cuda") / 999
        self.down, self.ds = torch.randint(-127, 128, (self.E, N, self.F), generator=gen, device="cuda", dtype=i8), torch.rand(self.E, N, generator=gen, device="cuda") / 999
        self.out = new(self.T, N, dtype=bf)

    def calls(self, h, i):
        B, M, N, K, fmt = V.IN_BF16, self.M, self.N, self.K, self.fmt
        yield lambda: self.route.copy_(self.ids[i % 3])
        yield lambda: V.sgemm_quantize_fp4(h, B, fmt, N, K, self.w[i % 2], K, self.qb, self.wide, self.sb, self.rb)
        yield lambda: V.sgemm_rms_norm_fp4(h, B, fmt, M, K, self.x[i % 3], K, self.residual, K, self.norm, EPS, self.residual, K, self.qa, self.wide, self.sa, self.ra)
        yield lambda: V.sgemm_run_fp4(h, fmt, B, M, N, K, self.qa, self.wide, self.sa, self.ra, self.qb, self.wide, self.sb, self.rb, None, self.y, N)
        yield lambda: V.sgemm_rms_norm_int8(h, B, M, N, self.y, N, None, 0, self.norm2, EPS, None, 0, self.q8, N, self.s8)
        yield lambda: V.sgemm_run_int8(h, 1, B, M, 96, N, self.q8, N, self.s8, self.b8, N, self.sb8, None, self.z, 96)
        yield lambda: V.sgemm_expert_layer_int8(h, B, 1, self.T, 2, self.E, N, self.F, self.y, N, self.route, self.cw, self.up, self.us, self.down, self.ds, self.out, N)

    def run(self, h, steps, wait=False, keep=True):
        self.residual.zero_()
        kept = []
        for i in range(steps):
            for call in self.calls(h, i):
                call()
                if wait:
                    torch.cuda.synchronize()
            if keep:
                kept += [self.y.clone(), self.z.clone(), self.out.clone(), self.residual.clone()]
        return kept


SIZES = [(5, 256, 640), (40, 330, 1001), (300, 512, 512), (700, 1000, 300)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_each_call_reads_what_the_one_before_wrote(g, fmt, M, N, K):
    s = Step(fmt, M, N, K, M)
    want = s.run(g.h, 12, wait=True)
    got = s.run(g.h, 12)
    torch.cuda.synchronize()
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES[:3])
def test_captured_and_replayed(g, fmt, M, N, K):
    """Two graphs of the same handle, replayed in turn (they share its workspace, in order)."""
    steps = [Step(fmt, M, N, K, 1), Step(fmt, max(1, M // 2), N, K, 2)]
    want = [[t.clone() for t in (s.run(g.h, 3, wait=True, keep=False), s.y, s.z, s.out)[1:]] for s in steps]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.run(g.h, 3, keep=False)
        graphs.append(graph)
    for _ in range(3):
        for s, graph, results in zip(steps, graphs, want):
            for t in (s.y, s.z, s.out):
                t.fill_(-3)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((s.y, s.z, s.out), results))


def test_gradient_captured_and_replayed(g):
    x, w = torch.randn(300, 1000, device="cuda"), torch.rand(1000, device="cuda")
    y, h, rstd = g.rms_norm(x, w)
    dy = torch.randn_like(x)
    want = g.rms_norm_grad(dy, x, w, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.rms_norm_grad(dy, x, w, rstd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = g.rms_norm_grad(dy, x, w, rstd)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- on another stream ------------------------------------------------------------------
def inputs(g):
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w, r = randn(96, 512).bfloat16(), randn(512).bfloat16(), randn(96, 512).bfloat16()
    a, b = g.quantize_fp4(x, V.FP4_NV), g.quantize_fp4(randn(256, 512), V.FP4_NV)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    return dict(x=x, w=w, r=r, aq=a.Q, as_=a.S, ar=a.row, bq=b.Q, bs=b.S, br=b.row, dy=randn(96, 512).bfloat16(), rstd=randn(96).abs(),
                ids=torch.randint(0, 4, (96, 2), generator=gen, device="cuda", dtype=torch.int32)[:40].contiguous(), weights=torch.rand(40, 2, generator=gen, device="cuda"),
                up=i8(4, 64, 512), us=randn(4, 64), down=i8(4, 512, 64), ds=randn(4, 512))


A = lambda d: V.Fp4Rows(d["aq"], d["as_"], d["ar"], 512, V.FP4_NV)  # noqa: E731
B = lambda d: V.Fp4Rows(d["bq"], d["bs"], d["br"], 512, V.FP4_NV)  # noqa: E731


def flat(result):
    return [t for r in tensors(result) for t in (r[:3] if isinstance(r, V.Fp4Rows) else (r,)) if torch.is_tensor(t)]


METHODS = {
    "quantize_fp4": lambda g, d, s: g.quantize_fp4(d["x"], V.FP4_NV, stream=s)[:3],
    "dequantize_fp4": lambda g, d, s: g.dequantize_fp4(A(d), stream=s),
    "matmul_fp4": lambda g, d, s: g.matmul_fp4(A(d), B(d), stream=s),
    "rms_norm": lambda g, d, s: g.rms_norm(d["x"], d["w"], d["r"], stream=s),
    "rms_norm_int8": lambda g, d, s: g.rms_norm_int8(d["x"], d["w"], d["r"], stream=s),
    "rms_norm_fp4": lambda g, d, s: g.rms_norm_fp4(d["x"], d["w"], d["r"], stream=s),
    "rms_norm_grad": lambda g, d, s: g.rms_norm_grad(d["dy"], d["x"], d["w"], d["rstd"], d["r"], stream=s),
    "expert_layer_int8": lambda g, d, s: g.expert_layer_int8(d["x"][:40], d["ids"], d["weights"], d["up"], d["us"], d["down"], d["ds"], stream=s),
}


def prepare(g, name):
    d, side = inputs(g), torch.cuda.Stream()
    torch.cuda.synchronize()
    METHODS[name](g, d, side)
    want = [t.clone() for t in flat(METHODS[name](g, d, None))]
    for t in (torch.empty_like(t) for t in (*want, *d.values())):
        t.fill_(77)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    return d, want, side


@pytest.mark.parametrize("name", list(METHODS))
def test_results_do_not_wait_for_or_mix_with_the_current_stream(g, name):
    d, want, side = prepare(g, name)
    torch.cuda._sleep(DELAY)
    freed = [torch.empty_like(t) for t in want]
    for t in freed:
        t.fill_(77)
    del freed, t
    got = flat(METHODS[name](g, d, side))
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was not busy any more: nothing was tested"
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", list(METHODS))
def test_inputs_stay_until_the_stream_has_read_them(g, name):
    d, want, side = prepare(g, name)
    sizes = [(t.shape, t.dtype) for t in d.values()]
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = flat(METHODS[name](g, d, side))
    d.clear()
    new = [torch.empty(shape, dtype=dtype, device="cuda").fill_(77) for shape, dtype in sizes]
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the side stream had read its inputs: nothing was tested"
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del new


# ---- refusals leave everything as it was -------------------------------------------------
def test_refused_calls_write_nothing_and_keep_the_report(g):
    h, t = g.h, torch.full((64, 64), 7.0, device="cuda")
    q, s = torch.full((4096,), 7, dtype=torch.uint8, device="cuda"), torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    i8, ids = torch.full((4096,), 7, dtype=torch.int8, device="cuda"), torch.zeros(64, 2, dtype=torch.int32, device="cuda")
    V.sgemm_run(h, 64, 64, 64, 1.0, t, 64, t, 64, 0.0, torch.zeros(64, 64, device="cuda"), 64)
    report = (*V.sgemm_last_variant(h), V.sgemm_last_launches(h))
    bad = [lambda: V.sgemm_quantize_fp4(h, 0, 0, 64, 64, t, 63, q, 32, s, None), lambda: V.sgemm_quantize_fp4(h, 0, 1, 64, 64, t, 64, q, 32, s, None),
           lambda: V.sgemm_quantize_fp4(h, 0, 0, 64, 64, t, 64, q, 32, s.data_ptr() + 8, None), lambda: V.sgemm_quantize_fp4(h, 0, 0, 64, 64, t, 64, t, 32, s, None),
           lambda: V.sgemm_quantize_fp4(h, 3, 0, 64, 64, t, 64, q, 32, s, None), lambda: V.sgemm_quantize_fp4(h, 0, 2, 64, 64, t, 64, q, 32, s, None),
           lambda: V.sgemm_dequantize_fp4(h, 0, 0, 64, 64, q, 31, s, None, t, 64), lambda: V.sgemm_dequantize_fp4(h, 0, 0, 64, 64, q, 32, None, None, t, 64),
           lambda: V.sgemm_run_fp4(h, 0, 0, 8, 8, 64, q, 32, s, None, q, 31, s, None, None, t, 64), lambda: V.sgemm_run_fp4(h, 1, 0, 8, 8, 64, q, 32, s, None, q, 32, s, None, None, t, 64),
           lambda: V.sgemm_rms_norm(h, 0, 8, 64, t, 64, t, 64, t, EPS, None, 0, t, 64, None), lambda: V.sgemm_rms_norm(h, 0, 8, 64, t, 64, None, 0, t[9], EPS, None, 0, t, 64, None),
           lambda: V.sgemm_rms_norm(h, 0, 8, 64, t, 64, None, 0, t[9], -1.0, None, 0, t[16:], 64, None), lambda: V.sgemm_rms_norm(h, 0, 8, 64, t, 64, None, 0, t[9], float("nan"), None, 0, t[16:], 64, None),
           lambda: V.sgemm_rms_norm(h, 0, 8, 64, t, 64, t[8:], 64, t[63], EPS, t[1:], 64, t[16:], 64, None),
           lambda: V.sgemm_rms_norm_int8(h, 0, 8, 64, t, 64, None, 0, t[9], EPS, None, 0, i8, 63, t[40]), lambda: V.sgemm_rms_norm_int8(h, 0, 8, 64, t, 64, None, 0, t[9], EPS, None, 0, i8, 64, None),
           lambda: V.sgemm_rms_norm_fp4(h, 0, 0, 8, 64, t, 64, None, 0, t[9], EPS, None, 0, q, 32, s, None), lambda: V.sgemm_rms_norm_grad(h, 0, 8, 64, t, 64, None, 0, t[8:], 64, t[20], t[21], t, 64, t[22]),
           lambda: V.sgemm_rms_norm_grad(h, 0, 8, 64, t, 64, None, 0, t[8:], 64, t[20], t[21], t[30:], 64, None), lambda: V.sgemm_rms_norm_grad(h, 0, 1, 12582913, t, 12582913, None, 0, t, 12582913, t, t, t, 12582913, t),
           lambda: V.sgemm_expert_layer_int8(h, 0, 0, 65, 2, 4, 64, 16, t, 64, ids, t, i8, t, i8, t, t, 64), lambda: V.sgemm_expert_layer_int8(h, 0, 2, 8, 2, 4, 64, 16, t, 64, ids, t, i8, t, i8, t, t[32:], 64),
           lambda: V.sgemm_expert_layer_int8(h, 0, 0, 64, 17, 4, 64, 16, t, 64, ids, t, i8, t, i8, t, t, 64), lambda: V.sgemm_expert_layer_int8(h, 0, 0, 8, 2, 1025, 64, 16, t, 64, ids, t, i8, t, i8, t, t, 64),
           lambda: V.sgemm_expert_layer_int8(h, 0, 0, 8, 2, 4, 64, 16, t, 63, ids, t, i8, t, i8, t, t, 64), lambda: V.sgemm_expert_layer_int8(h, 0, 0, 8, 2, 4, 64, 16, t, 64, ids, None, i8, t, i8, t, t, 64),
           lambda: V.sgemm_expert_layer_int8(h, 0, 0, 8, 2, 4, 64, 16, t, 64, ids, t[60], i8, t[50], i8, t[55], t, 64), lambda: V.sgemm_expert_layer_int8(h, 0, 0, 64, 16, 4, 64, 1 << 24, t, 64, ids, t, i8, t, i8, t, t, 64)]
    for i, call in enumerate(bad):
        with pytest.raises(sgemm.SgemmError) as e:
            call()
        assert e.value.status in (V.ERR_NULL, V.ERR_INVALID_VALUE, V.ERR_ALIAS), i
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in (t, q, s, i8))
    assert (*V.sgemm_last_variant(h), V.sgemm_last_launches(h)) == report
    V.sgemm_quantize_fp4(h, 0, 0, 64, 64, t, 64, q, 32, s, None)
    assert (*V.sgemm_last_variant(h), V.sgemm_last_launches(h)) == (-1, 1, 1)
    V.sgemm_rms_norm(h, 0, 0, 64, None, 64, None, 0, None, EPS, None, 0, None, 64, None)
    assert V.sgemm_last_launches(h) == 0


# ---- buffers past 2^31 elements -----------------------------------------------------------
def test_wide_offsets(g):
    """2^31 elements and some: sampled rows alone are compared, with what the same rows give in a small
    call (which the other tests hold to the definition)."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("too little free memory")
    K, rows = 8192, (1 << 31) // 8192 + 4099
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 65536):
        x[r:r + 65536] = torch.randn(min(65536, rows - r), K, generator=gen, device="cuda")
    w = (1 + torch.randn(K, generator=gen, device="cuda") / 5).bfloat16()
    at = torch.tensor([0, 1, 12345, rows - 1, rows - 2, (1 << 31) // K, (1 << 31) // K - 1, (1 << 30) // K + 7], device="cuda")
    few = x[at].contiguous()
    q, scale, _ = g.rms_norm_int8(x, w)
    q1, scale1, _ = g.rms_norm_int8(few, w)
    assert torch.equal(q[at], q1) and bool(((scale[at] - scale1).abs() <= 1e-5 * scale1).all())
    del q, scale
    b = g.quantize_fp4(torch.randn(72, K, generator=gen, device="cuda"), V.FP4_NV)
    rows4, few4 = g.quantize_fp4(x, V.FP4_NV), g.quantize_fp4(few, V.FP4_NV)
    assert torch.equal(rows4.Q[at], few4.Q) and torch.equal(rows4.row[at], few4.row)
    got, want = g.matmul_fp4(rows4, b, out_dtype=torch.float32)[at], g.matmul_fp4(few4, b, out_dtype=torch.float32)
    assert bool(((got - want).abs() <= 1e-5 * want.abs().max()).all())
    # rows on no boundary are copied (in the workspace they do not fit: the generic kernel)
    odd = rows4._replace(Q=torch.nn.functional.pad(rows4.Q, (0, 3)))
    out = g.matmul_fp4(odd, b, out_dtype=torch.float32)
    assert g.last_variant[0] == V.VARIANT_GENERIC_F4
    assert bool(((out[at] - want).abs() <= 1e-5 * want.abs().max()).all())
    del odd, out
    back = g.dequantize_fp4(rows4)
    assert torch.equal(back[at], g.dequantize_fp4(few4))
    del back, rows4
    y, _, rstd = g.rms_norm(x, w)
    y1, _, rstd1 = g.rms_norm(few, w)
    assert bool(((rstd[at] - rstd1).abs() <= 1e-5 * rstd1).all()) and bool(((y[at].float() - y1.float()).abs() <= 2.0 ** -7 * y1.float().abs()).all())
    dx, _ = g.rms_norm_grad(y, x, w, rstd)
    dx1, _ = g.rms_norm_grad(y[at].contiguous(), few, w, rstd[at].contiguous())
    assert torch.equal(dx[at], dx1)


# ---- the example --------------------------------------------------------------------------
def test_the_norm_as_a_function_of_autograd(g):
    """Gradients of (norm(x + r) w, x + r) against torch's in 64 bits: sums of 96 terms and a few roundings
    in FP32, 1e-5 of the norm."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, r, w = (torch.randn(*s, generator=gen, device="cuda") for s in ((33, 96), (33, 96), (96,)))
    params = [t.clone().requires_grad_() for t in (x, r, w)]
    y, h = ex.Norm.apply(*params, EPS, g)
    exact = [t.double().requires_grad_() for t in (x, r, w)]
    eh = exact[0] + exact[1]
    ey = eh / (eh.square().mean(1, keepdim=True) + EPS).sqrt() * exact[2]
    cy, ch = torch.randn(33, 96, generator=gen, device="cuda"), torch.randn(33, 96, generator=gen, device="cuda")
    ((y * cy).sum() + (h * ch).sum()).backward()
    ((ey * cy).sum() + (eh * ch).sum()).backward()
    for p, e in zip(params, exact):
        assert float((p.grad - e.grad).norm()) <= 1e-5 * float(e.grad.norm())
    y, h = ex.Norm.apply(*params, EPS, g)     # the residual's way alone: no gradient reaches y
    params[2].grad = None
    (h * ch).sum().backward()
    assert bool((params[2].grad == 0).all())


def test_the_example_runs(g, capsys):
    ex.main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 5


@pytest.mark.parametrize("tokens,dropped", [(1, False), (7, True), (64, True)])
def test_few_tokens_served_in_two_launches(g, tokens, dropped):
    """Weights in 8 bits (two operands of the four that test_served counts): within the same 5 %."""
    from tests.test_gpu_expert_layer import layer
    x, ids, weights, up, down = layer(tokens, 128, 96, 6, 2, dropped)
    want = ex.plain_forward(x.double(), ids, weights.double(), up.double(), down.double())
    got = ex.ServedExperts(g, up, down).few(x.bfloat16(), ids, weights)
    assert g.h is not None and V.sgemm_last_launches(g.h) == 2
    assert float((got.double() - want).norm()) <= 0.05 * float(want.norm())


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_and_product_in_4_bits_are_those_of_what_the_rows_stand_for(g, fmt):
    """The layer's result is the product of the values that its 4-bit rows stand for, whose
    row scales carry 1 / rms: (K + 3) 2^-23 of the terms' magnitudes and BF16's half step."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, r = (torch.randn(50, 300, generator=gen, device="cuda").bfloat16() for _ in range(2))
    norm, matrix = (1 + torch.randn(300, generator=gen, device="cuda") / 9).bfloat16(), torch.randn(70, 300, generator=gen, device="cuda").bfloat16()
    y, h = ex.ServedLinear(g, norm, matrix, fmt)(x, r)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    rows, _ = g.rms_norm_fp4(x, norm, r, EPS, fmt)
    a = f4.values(fmt, f4.unpack(rows.Q.cpu(), 300), rows.S.cpu()[f4.scale_index(fmt, 50, 300)], rows.row.cpu())
    b4 = g.quantize_fp4(matrix, fmt)
    b = f4.values(fmt, f4.unpack(b4.Q.cpu(), 300), b4.S.cpu()[f4.scale_index(fmt, 70, 300)], b4.row.cpu() if b4.row is not None else None)
    want, size = a @ b.T, a.abs() @ b.abs().T
    err = 303 * 2.0 ** -23 * size
    assert ((y.cpu().double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all()
