"""The whole expert layer for a few tokens against a 64-bit form.

Tolerance: a hidden value's sum over `width` terms is off by at most (width + 3) u of the
terms' magnitudes (u = 2^-23: a tensor core's sum may truncate; the int8 and the
tokens' parts are exact; FP32 tokens leave out the products below 2^-24 of theirs); silu's slope is at
most 1.1 and the factor, product and roundings of it add 8 u; kept in 16 (24) bits, another 2^-16
(2^-24).  The sum over the hidden values and the choices likewise, (hidden + 8 + choices) u,
the rounding to the type at the end."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm

pytestmark = pytest.mark.gpu

TYPES = {sgemm.IN_F32: torch.float32, sgemm.IN_BF16: torch.bfloat16, sgemm.IN_F16: torch.float16}
U = 2.0 ** -23


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


def reference(x, ids, weights, up, us, down, ds, gated):
    """(out, bound of the FP32 errors)."""
    x, us, ds, weights = x.double(), us.double(), ds.double(), weights.double()
    E, F, W = up.shape[0], down.shape[2], down.shape[1]
    out, err = torch.zeros(x.shape[0], W, dtype=torch.float64), torch.zeros(x.shape[0], W, dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            U_, D_ = up[e].double(), down[e].double()
            y, size = (U_ @ x[t]) * us[e], (U_.abs() @ x[t].abs()) * us[e]
            dy = (W + 3) * U * size
            a = y[:F] / (1 + torch.exp(-y[:F]))
            da = 1.1 * dy[:F] + 8 * U * a.abs()
            if gated:
                da = da * y[F:].abs() + (a.abs() + da) * dy[F:] + U * (a * y[F:]).abs()
                a = a * y[F:]
            w = weights[t, j]
            out[t] += w * (D_ @ a) * ds[e]
            err[t] += w.abs() * ds[e] * (D_.abs() @ da + D_.abs() @ a.abs() * (F + 8 + ids.shape[1]) * U)
            err[t] += w.abs() * ds[e] * (D_.abs() @ a.abs()) * (2.0 ** -24 if x.dtype == torch.float32 else 2.0 ** -16)
    return out, err


def problem(kind, gated, T, J, E, W, F, seed=0, ids=None):
    g = torch.Generator().manual_seed(seed + 100 * T + W + F)
    x = (torch.randn(T, W, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g))).to(TYPES[kind])
    if ids is None:
        ids = torch.rand(T, E, generator=g).topk(min(J, E), dim=1).indices
        if J > E:
            ids = torch.cat((ids, torch.randint(0, E, (T, J - E), generator=g)), dim=1)
    ids = ids.to(torch.int32).contiguous()
    weights = torch.softmax(torch.randn(T, J, generator=g), dim=1).contiguous()
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8)  # noqa: E731
    up, us = i8(E, (2 if gated else 1) * F, W), (0.5 + torch.rand(E, (2 if gated else 1) * F, generator=g)) / (74 * max(W, 1) ** 0.5)
    down, ds = i8(E, W, F), (0.5 + torch.rand(E, W, generator=g)) / (74 * max(F, 1) ** 0.5)
    return x, ids, weights, up, us, down, ds


def run(h, kind, gated, p, pad=0, off=0):
    x, ids, weights, up, us, down, ds = p
    (T, W), J, E, F = x.shape, ids.shape[1], up.shape[0], down.shape[2]
    X = torch.full((off + T * (W + pad) + 8,), 99.0, dtype=x.dtype)
    X[off:off + T * (W + pad)].view(T, W + pad)[:, :W] = x
    X = X.cuda()
    out = torch.full((T + 1, W + pad), 7.0, dtype=x.dtype, device="cuda")
    def shifted(t):
        full = torch.full((t.numel() + off,), 5, dtype=t.dtype, device="cuda")
        full[off:] = t.reshape(-1).cuda()
        return full[off:]
    dev = [ids.cuda(), weights.cuda(), shifted(up), us.cuda(), shifted(down), ds.cuda()]
    sgemm.sgemm_expert_layer_int8(h, kind, int(gated), T, J, E, W, F, X[off:], W + pad, *dev, out, W + pad)
    torch.cuda.synchronize()
    got = out.cpu()
    assert (got[T] == 7).all() and (got[:, W:] == 7).all()
    return got[:T, :W]


def check(h, kind, gated, p, **more):
    got = run(h, kind, gated, p, **more)
    want, err = reference(*p, gated)
    dtype = TYPES[kind]
    t, tiny = torch.finfo(dtype).eps / 2, float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    bad = ((got.double() - want).abs() > err + t * (want.abs() + err) + tiny).nonzero()
    assert not len(bad), (len(bad), bad[0].tolist(), float(got[tuple(bad[0])]), float(want[tuple(bad[0])]))
    return got


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", [(1, 1, 1, 64, 64), (1, 4, 8, 256, 128), (8, 2, 4, 128, 192), (9, 2, 4, 128, 64), (33, 1, 2, 64, 80), (64, 4, 8, 256, 96),
                                       (64, 2, 2, 128, 64), (5, 16, 40, 64, 64), (3, 2, 1024, 64, 16), (64, 16, 16, 64, 64)])
def test_layer(h, kind, gated, T, J, E, W, F):
    check(h, kind, gated, problem(kind, gated, T, J, E, W, F))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", [(1, 2, 3, 1, 1), (2, 1, 2, 7, 5), (5, 3, 4, 65, 33), (17, 2, 4, 100, 130), (12, 2, 3, 301, 77), (64, 2, 4, 48, 1000)])
def test_odd_sizes_and_addresses(h, kind, gated, T, J, E, W, F):
    p = problem(kind, gated, T, J, E, W, F)
    check(h, kind, gated, p)
    check(h, kind, gated, p, pad=3, off=1)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", [(8, 2, 3, 2448, 80), (5, 1, 1, 4096, 1040), (1, 3, 5, 4880, 64), (8, 1, 1, 6992, 144), (8, 4, 9, 2560, 2064), (8, 3, 4, 9744, 16)])
def test_wide_rows_of_a_few_tokens(h, kind, gated, T, J, E, W, F):
    """More channels than 16 an SM: items of up to 32, the last one cut, one round or more of them; experts
    of one column and of all eight."""
    check(h, kind, gated, problem(kind, gated, T, J, E, W, F))


@pytest.mark.parametrize("T", [4, 40])
def test_dropped_repeated_and_crowded_choices(h, T):
    J, E, W, F = 3, 5, 96, 64
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-2, E + 2, (T, J), generator=g)
    ids[0] = torch.tensor([2, 2, 2])            # the same expert three times
    ids[1] = torch.tensor([-1, E, 1 << 30])     # none at all
    ids[2] = torch.tensor([4, -5, 4])
    for kind in TYPES:
        got = check(h, kind, True, problem(kind, True, T, J, E, W, F, ids=ids))
        assert (got[1] == 0).all()
    check(h, sgemm.IN_BF16, True, problem(sgemm.IN_BF16, True, T, J, E, W, F, ids=torch.zeros(T, J) + torch.tensor([3, 9, 9])))
    nobody = run(h, sgemm.IN_BF16, False, problem(sgemm.IN_BF16, False, T, J, E, W, F, ids=torch.full((T, J), -1)))
    assert (nobody == 0).all()


def test_no_hidden_channels(h):
    assert (run(h, sgemm.IN_F32, True, problem(sgemm.IN_F32, True, 3, 2, 4, 32, 0)) == 0).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_same_bits_every_time(h, kind):
    p = problem(kind, True, 8, 2, 4, 512, 256)
    first = run(h, kind, True, p)
    for _ in range(3):
        assert torch.equal(run(h, kind, True, p), first)


def test_as_the_chain_of_calls(h):
    """sort, dispatch in 8 bits, two int8 products, combine: the same layer but for the tokens' and the
    hidden values' rounding to 8 bits, which is off by half a step of 1/127 of a row's largest value in
    either product; with rows of normal values that is 2^-8 of a value's typical size, so the results
    are apart by a few percent at most."""
    T, J, E, W, F = 16, 2, 4, 256, 512
    x, ids, weights, up, us, down, ds = problem(sgemm.IN_BF16, False, T, J, E, W, F)
    whole = run(h, sgemm.IN_BF16, False, (x, ids, weights, up, us, down, ds)).double()
    with sgemm.Sgemm() as g:
        d = [t.cuda() for t in (x, ids, weights, up, us, down, ds)]
        offsets, rows, _ = g.expert_sort(d[1], E)
        q, s = g.expert_dispatch_int8(d[0], rows)
        hid = g.matmul_int8_experts(offsets, q, s, d[3], d[4], out_dtype=torch.float32)
        q, s = g.quantize(torch.nn.functional.silu(hid))
        y = g.matmul_int8_experts(offsets, q, s, d[5], d[6], out_dtype=torch.bfloat16)
        chain = g.expert_combine(y, rows, d[2]).cpu().double()
    assert float((whole - chain).norm() / chain.norm()) < 0.05
