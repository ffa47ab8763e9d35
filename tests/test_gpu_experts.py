"""GPU parity of the expert routing calls (sgemm_expert_*) against plain
64-bit forms.

Tolerances: copies and integers are equal.  A sum over J choices in FP32 with
fused multiply-adds errs by at most J * 2^-24 * sum |w y| (J roundings, one a
step; (1 + 2^-24)^J - 1 < 1.01 J 2^-24 here), then the rounding to the type:
u |exact|, u = 2^-24, 2^-8, 2^-11 (2^-p for p significant bits; + 2^-25 for
FP16's subnormals).  dY is one
product, rounded in FP32 and again to the type.  A dot product over `width`
elements errs by at most D * 2^-24 * sum |dO Y|, D the longest chain of
additions: every 2048th element in a thread's fused chain, 8 a step
(ceil(width / 2048) * 8), 5 steps within the warp, 8 warps."""
import math

import numpy as np
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import TYPES, addr, plain_quantize, strided

pytestmark = pytest.mark.gpu

V = sgemm
EPS = 2.0 ** -24


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


def plain_sort(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    kept = int(offsets[-1])
    rows = np.full(flat.size, -1)
    rows[order[:kept]] = np.arange(kept)
    source = np.full(flat.size, -1)
    source[:kept] = order[:kept]
    return offsets, rows, source


def gpu_sort(h, ids, experts):
    tokens, choices = ids.shape
    n = tokens * choices
    d = torch.from_numpy(ids.astype(np.int32)).cuda()
    off = torch.full((experts + 2,), -7, dtype=torch.int32, device="cuda")
    rows, source = (torch.full((n + 1,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sgemm.sgemm_expert_sort(h, tokens, choices, experts, d, off, rows, source)
    torch.cuda.synchronize()
    assert int(off[-1]) == int(rows[-1]) == int(source[-1]) == -7
    return off[:-1], rows[:-1], source[:-1]


def make_ids(tokens, choices, experts, kind, seed=0):
    rng = np.random.default_rng(seed + tokens * 13 + experts)
    ids = rng.integers(0, experts, (tokens, choices))
    if kind == "one":
        ids[:] = experts - 1
    elif kind == "dropped":
        ids[rng.random(ids.shape) < 0.3] = -1
        ids[rng.random(ids.shape) < 0.1] = experts
        ids.flat[0] = -2 ** 31
        ids.flat[-1] = 2 ** 31 - 1
    elif kind == "none":
        ids[:] = -1
    return ids


@pytest.mark.parametrize("tokens,choices,experts", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (32, 4, 32), (255, 1, 7),
                                                    (257, 1, 300), (1000, 4, 128), (1024, 4, 1024), (1025, 4, 16),
                                                    (5000, 3, 1000), (40000, 8, 60), (1 << 20, 1, 8)])
@pytest.mark.parametrize("kind", ["even", "one", "dropped", "none"])
def test_sort(handle, tokens, choices, experts, kind):
    ids = make_ids(tokens, choices, experts, kind)
    for got, want in zip(gpu_sort(handle, ids, experts), plain_sort(ids, experts)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_of_nothing_and_refusals(handle):
    off = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    sgemm.sgemm_expert_sort(handle, 0, 2, 8, None, off, None, None)
    torch.cuda.synchronize()
    assert off.tolist() == [0] * 9
    ids, rows, src = (torch.zeros(16, dtype=torch.int32, device="cuda") for _ in range(3))

    def status(**k):
        d = dict(tokens=4, choices=2, experts=8, ids=ids, offsets=off, rows=rows, source=src)
        d.update(k)
        try:
            sgemm.sgemm_expert_sort(handle, **d)
        except sgemm.SgemmError as e:
            return e.status
        return V.OK

    assert status() == V.OK
    for bad in (dict(tokens=-1), dict(choices=0), dict(experts=0), dict(experts=1025), dict(tokens=2 ** 30, choices=2),
                dict(ids=ids.data_ptr() + 1)):
        assert status(**bad) == V.ERR_INVALID_VALUE, bad
    for bad in (dict(ids=None), dict(offsets=None), dict(rows=None), dict(source=None)):
        assert status(**bad) == V.ERR_NULL, bad
    assert status(rows=ids) == V.ERR_ALIAS
    assert status(source=rows) == V.ERR_ALIAS
    torch.cuda.synchronize()


SHAPES = [(1, 1, 1), (5, 2, 33), (9, 4, 64), (33, 3, 1000), (64, 8, 256), (300, 2, 2056), (17, 5, 4099), (2, 9, 8192)]


class Routed:
    """tokens, the sorted rows of their slots (some dropped) and buffers with odd strides."""

    def __init__(self, h, tokens, choices, width, dtype, pad, offset, kind="dropped"):
        self.g = torch.Generator().manual_seed(tokens * 7 + width)
        self.T, self.J, self.W, self.kind, self.type = tokens, choices, width, *TYPES[dtype][:2]
        self.u = max(TYPES[dtype][2], EPS)
        self.tiny = 2.0 ** -25 if dtype == "f16" else 0.0
        self.pad, self.offset, self.slots = pad, offset, tokens * choices
        ids = make_ids(tokens, choices, 6, kind)
        self.rows = gpu_sort(h, ids, 6)[1]
        self.r = self.rows.cpu().numpy()
        self.kept = np.nonzero(self.r >= 0)[0]

    def buf(self, rows, fill=None):
        x = torch.randn(rows, self.W, generator=self.g) if fill is None else torch.full((rows, self.W), fill)
        return strided(x.to(self.type), self.pad, self.offset, fill=fill if fill is not None else 1e4)

    def p(self, b):
        return addr(*b, self.offset)

    @property
    def ld(self):
        return self.W + self.pad

    def double(self, b):
        return b[0].cpu().double().numpy()

    def untouched(self, b, fill, rows):
        """Only the window's `rows` of b may have changed from fill."""
        full = b[1].clone()
        n = b[0].shape[0] * self.ld
        full[self.offset:self.offset + n].view(-1, self.ld)[torch.as_tensor(rows, device="cuda"), :self.W] = fill
        assert bool((full == fill).all())


LAYOUTS = [(0, 0), (8, 8), (1, 3)]


@pytest.mark.parametrize("tokens,choices,width", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", LAYOUTS)
def test_dispatch_and_its_gradient(handle, tokens, choices, width, dtype, pad, offset):
    t = Routed(handle, tokens, choices, width, dtype, pad, offset)
    x, y = t.buf(tokens), t.buf(t.slots, 9.0)
    sgemm.sgemm_expert_dispatch(handle, t.kind, tokens, choices, width, t.p(x), t.ld, t.rows, t.p(y), t.ld)
    dy, dx = t.buf(t.slots), t.buf(tokens, 9.0)
    dy[0][torch.as_tensor(np.setdiff1d(np.arange(t.slots), t.r[t.kept]), device="cuda")] = float("nan")  # unused rows
    sgemm.sgemm_expert_dispatch_grad(handle, t.kind, tokens, choices, width, t.p(dy), t.ld, t.rows, t.p(dx), t.ld)
    torch.cuda.synchronize()
    got = y[0].cpu()
    assert torch.equal(got[t.r[t.kept]], x[0].cpu()[t.kept // choices])
    t.untouched(y, 9.0, t.r[t.kept])
    want, mag = np.zeros((tokens, width)), np.zeros((tokens, width))
    d = t.double(dy)
    for s in t.kept:
        want[s // choices] += d[t.r[s]]
        mag[s // choices] += np.abs(d[t.r[s]])
    tol = 1.01 * choices * EPS * mag + t.u * np.abs(want) * (1 + 2.0 ** -20) + t.tiny
    assert np.all(np.abs(t.double(dx) - want) <= tol)
    t.untouched(dx, 9.0, np.arange(tokens))


@pytest.mark.parametrize("tokens,choices,width", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_dispatch_int8_is_the_quantized_dispatch(handle, tokens, choices, width, dtype):
    t = Routed(handle, tokens, choices, width, dtype, 3, 1)
    x = t.buf(tokens)
    if tokens > 2:
        x[0][1] = 0
        x[0][2, 0] = float("inf")
    q, qf = strided(torch.full((t.slots, width), 99, dtype=torch.int8), 5, 1, fill=99)
    scale = torch.full((t.slots,), -1.0, device="cuda")
    sgemm.sgemm_expert_dispatch_int8(handle, t.kind, tokens, choices, width, t.p(x), t.ld, t.rows, addr(q, qf, 1),
                                     width + 5, scale)
    torch.cuda.synchronize()
    want_q, want_s = plain_quantize(x[0].cpu())
    got_q, got_s = q.cpu().numpy(), scale.cpu().numpy()
    assert np.array_equal(got_q[t.r[t.kept]], want_q[t.kept // choices])
    assert np.array_equal(got_s[t.r[t.kept]], want_s[t.kept // choices], equal_nan=True)
    rest = np.setdiff1d(np.arange(t.slots), t.r[t.kept])
    assert np.all(got_q[rest] == 99) and np.all(got_s[rest] == -1)


@pytest.mark.parametrize("tokens,choices,width", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", LAYOUTS)
def test_combine_and_its_gradients(handle, tokens, choices, width, dtype, pad, offset):
    t = Routed(handle, tokens, choices, width, dtype, pad, offset)
    y, out, dout, dy = t.buf(t.slots), t.buf(tokens, 9.0), t.buf(tokens), t.buf(t.slots, 9.0)
    y[0][torch.as_tensor(np.setdiff1d(np.arange(t.slots), t.r[t.kept]), device="cuda")] = float("nan")  # unused rows
    w = torch.rand(tokens, choices, generator=t.g)
    for s in np.setdiff1d(np.arange(t.slots), t.kept):
        w.view(-1)[s] = float("nan")                       # a dropped slot's weight is not used
    W, dw = w.cuda(), torch.full((t.slots + 1,), -7.0, device="cuda")
    sgemm.sgemm_expert_combine(handle, t.kind, tokens, choices, width, t.p(y), t.ld, t.rows, W, t.p(out), t.ld)
    sgemm.sgemm_expert_combine_grad(handle, t.kind, tokens, choices, width, t.p(dout), t.ld, t.p(y), t.ld, t.rows, W,
                                    t.p(dy), t.ld, dw)
    torch.cuda.synchronize()
    yd, gd, wd = t.double(y), t.double(dout), w.double().numpy().reshape(-1)
    want, mag = np.zeros((tokens, width)), np.zeros((tokens, width))
    want_dw, mag_dw = np.zeros(t.slots), np.zeros(t.slots)
    for s in t.kept:
        want[s // choices] += wd[s] * yd[t.r[s]]
        mag[s // choices] += np.abs(wd[s] * yd[t.r[s]])
        want_dw[s] = np.dot(gd[s // choices], yd[t.r[s]])
        mag_dw[s] = np.dot(np.abs(gd[s // choices]), np.abs(yd[t.r[s]]))
    tol = 1.01 * choices * EPS * mag + t.u * np.abs(want) * (1 + 2.0 ** -20) + t.tiny
    assert np.all(np.abs(t.double(out) - want) <= tol)
    t.untouched(out, 9.0, np.arange(tokens))
    chain = math.ceil(width / 2048) * 8 + 5 + 8
    assert np.all(np.abs(dw[:-1].cpu().double().numpy() - want_dw) <= 1.01 * chain * EPS * mag_dw)
    assert float(dw[-1]) == -7.0
    want_dy = wd[t.kept, None] * gd[t.kept // choices]
    got_dy = t.double(dy)[t.r[t.kept]]
    assert np.all(np.abs(got_dy - want_dy) <= (EPS + t.u * (1 + 2.0 ** -20)) * np.abs(want_dy) + t.tiny)
    t.untouched(dy, 9.0, t.r[t.kept])


def test_gradients_against_differences(handle):
    """L = sum(out * dout) is linear in Y and in the weights apart, so a central
    difference with step 1 is the derivative up to the rounding of the two forward
    passes: each out errs by (J + 1) * 2^-24 * sum |w y| (width of them, summed in
    64 bits here), and the analytic gradient by its own bound."""
    T, J, W = 6, 3, 40
    t = Routed(handle, T, J, W, "f32", 0, 0, kind="even")
    y, dout, dy, out = t.buf(t.slots), t.buf(T), t.buf(t.slots, 0.0), t.buf(T, 0.0)
    w = torch.rand(T, J, generator=t.g).cuda()
    dw = torch.zeros(t.slots, device="cuda")
    sgemm.sgemm_expert_combine_grad(handle, t.kind, T, J, W, t.p(dout), W, t.p(y), W, t.rows, w, t.p(dy), W, dw)

    def loss():
        sgemm.sgemm_expert_combine(handle, t.kind, T, J, W, t.p(y), W, t.rows, w, t.p(out), W)
        torch.cuda.synchronize()
        return float((out[0].double() * dout[0].double()).sum())

    # |w| <= 2, |y| < 6, |dout| < 6 after the step: every term's rounding, over all outputs
    bound = 2 * T * W * 6 * (J + 1) * EPS * J * 2 * 7
    for slot in range(0, t.slots, 4):
        w.view(-1)[slot] += 1
        up = loss()
        w.view(-1)[slot] -= 2
        down = loss()
        w.view(-1)[slot] += 1
        assert abs((up - down) / 2 - float(dw[slot])) <= bound
        r = int(t.r[slot])
        for p in (0, 17, 39):
            y[0][r, p] += 1
            up = loss()
            y[0][r, p] -= 2
            down = loss()
            y[0][r, p] += 1
            assert abs((up - down) / 2 - float(dy[0][r, p])) <= bound


def test_dispatch_gradient_against_differences(handle):
    """As above: L = sum(Y * dY) is linear in X and dispatch copies, so the difference errs only by FP32's x + 1 - 1."""
    T, J, W = 5, 2, 24
    t = Routed(handle, T, J, W, "f32", 0, 0, kind="dropped")
    x, y, dy, dx = t.buf(T), t.buf(t.slots, 0.0), t.buf(t.slots), t.buf(T, 0.0)
    sgemm.sgemm_expert_dispatch_grad(handle, t.kind, T, J, W, t.p(dy), W, t.rows, t.p(dx), W)

    def loss():
        sgemm.sgemm_expert_dispatch(handle, t.kind, T, J, W, t.p(x), W, t.rows, t.p(y), W)
        torch.cuda.synchronize()
        return float((y[0].double()[t.r[t.kept]] * dy[0].double()[t.r[t.kept]]).sum())

    for token in range(T):
        for p in (0, 11, 23):
            x[0][token, p] += 1
            up = loss()
            x[0][token, p] -= 2
            down = loss()
            x[0][token, p] += 1
            assert abs((up - down) / 2 - float(dx[0][token, p])) <= 8 * EPS * J * 8 * 2


def test_rows_out_of_range_are_dropped_slots(handle):
    rows = torch.tensor([0, 99, -5, 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    x = torch.arange(24, dtype=torch.float32, device="cuda").view(3, 8)
    y = torch.full((7, 8), -1.0, device="cuda")
    sgemm.sgemm_expert_dispatch(handle, V.IN_F32, 3, 2, 8, x, 8, rows, y, 8)
    w, out = torch.ones(6, device="cuda"), torch.zeros(3, 8, device="cuda")
    sgemm.sgemm_expert_combine(handle, V.IN_F32, 3, 2, 8, y, 8, rows, w, out, 8)
    torch.cuda.synchronize()
    assert torch.equal(y[0], x[0]) and torch.equal(y[3], x[1])
    assert bool((y[[1, 2, 4, 5, 6]] == -1).all())
    assert torch.equal(out[:2], x[:2]) and bool((out[2] == 0).all())


CALLS = {
    "dispatch": (sgemm.sgemm_expert_dispatch, ["X", "ldx", "rows", "Y", "ldy"], "Y"),
    "dispatch_grad": (sgemm.sgemm_expert_dispatch_grad, ["dY", "lddy", "rows", "dX", "lddx"], "dX"),
    "dispatch_int8": (sgemm.sgemm_expert_dispatch_int8, ["X", "ldx", "rows", "Q", "ldq", "scale"], "Q"),
    "combine": (sgemm.sgemm_expert_combine, ["Y", "ldy", "rows", "weights", "out", "ldo"], "out"),
    "combine_grad": (sgemm.sgemm_expert_combine_grad,
                     ["dout", "lddo", "Y", "ldy", "rows", "weights", "dY", "lddy", "dweights"], "dY"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(handle, name):
    call, names, output = CALLS[name]
    bufs = {n: torch.zeros(256, dtype=torch.int8 if n == "Q" else torch.int32 if n == "rows" else torch.float32,
                           device="cuda") for n in names if not n.startswith("ld")}

    def status(**k):
        d = dict(in_type=V.IN_F32, tokens=3, choices=2, width=16)
        for n in names:
            d[n] = 16 if n.startswith("ld") else bufs[n]
        d.update(k)
        try:
            call(handle, **d)
        except sgemm.SgemmError as e:
            return e.status
        return V.OK

    assert status() == V.OK
    assert status(tokens=0) == V.OK
    for bad in [dict(in_type=5), dict(tokens=-1), dict(choices=0), dict(width=-1), dict(tokens=2 ** 30, choices=4)] + \
            [{n: 15} for n in names if n.startswith("ld")] + \
            [{n: bufs[n].data_ptr() + 1} for n in bufs if n != "Q"]:
        assert status(**bad) == V.ERR_INVALID_VALUE, bad
    for n in bufs:
        assert status(**{n: None}) == V.ERR_NULL, n
    for n in bufs:
        if n != output:
            assert status(**{output: bufs[n]}) == V.ERR_ALIAS, n
    try:
        call(None, **{**dict(in_type=0, tokens=3, choices=2, width=16),
                      **{n: 16 if n.startswith("ld") else bufs[n] for n in names}})
        raise AssertionError("a NULL handle was accepted")
    except sgemm.SgemmError as e:
        assert e.status == V.ERR_BAD_HANDLE
    torch.cuda.synchronize()
