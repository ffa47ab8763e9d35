"""The whole expert layer on rows and hidden values of several kilobytes, with any number of tokens:
every loop of its kernels makes more than one round.  Then what a token or a choice
with an infinity or a NaN leaves alone, and inputs that the kernel right before wrote.

Reference and bound as in test_gpu_expert_layer_few, an expert's tokens at a time."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_expert_layer_few import TYPES, U, problem, run
from tests.test_gpu_expert_layer_few import h  # noqa: F401  (the handle)

pytestmark = pytest.mark.gpu


def reference(x, ids, weights, up, us, down, ds, gated):
    """(out, bound of the FP32 errors), in 64 bits."""
    kept = 2.0 ** -24 if x.dtype == torch.float32 else 2.0 ** -16
    x, us, ds, weights, ids = x.cuda().double(), us.cuda().double(), ds.cuda().double(), weights.cuda().double(), ids.cuda()
    (E, W, F), J = down.shape, ids.shape[1]
    out = torch.zeros(x.shape[0], W, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        U_, D_ = up[e].cuda().double(), down[e].cuda().double()
        y, size = x[t] @ U_.T * us[e], x[t].abs() @ U_.abs().T * us[e]
        dy = (W + 3) * U * size
        a = y[:, :F] / (1 + torch.exp(-y[:, :F]))
        da = 1.1 * dy[:, :F] + 8 * U * a.abs()
        if gated:
            da = da * y[:, F:].abs() + (a.abs() + da) * dy[:, F:] + U * (a * y[:, F:]).abs()
            a = a * y[:, F:]
        w = weights[t, j][:, None]
        sums = a.abs() @ D_.abs().T
        out.index_add_(0, t, w * (a @ D_.T) * ds[e])
        err.index_add_(0, t, w.abs() * ds[e] * (da @ D_.abs().T + sums * ((F + 8 + J) * U + kept)))
    return out.cpu(), err.cpu()


def compare(got, want, err, rows=slice(None)):
    t, tiny = torch.finfo(got.dtype).eps / 2, float(torch.finfo(got.dtype).smallest_normal) * torch.finfo(got.dtype).eps
    bad = ((got[rows].double() - want[rows]).abs() > err[rows] + t * (want[rows].abs() + err[rows]) + tiny).nonzero()
    assert not len(bad), (len(bad), bad[0].tolist())


def check(h, kind, gated, p, **more):  # noqa: F811
    got = run(h, kind, gated, p, **more)
    want, err = reference(*p, gated)
    compare(got, want, err)
    # That bound is of the worst case.  On the whole: 16-bit results at most half a step each; FP32 ones half
    # a truncation, 2^-24, for each of a chain's MMAs (16 terms of three parts), 16 more for what is around them.
    W, F = p[0].shape[1], p[5].shape[2]
    whole = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else (3 * (W + F) / 16 + 16) * 2.0 ** -24
    assert float((got.double() - want).norm()) <= whole * float(want.norm())
    return got


def test_the_two_references_agree():
    from tests.test_gpu_expert_layer_few import reference as one_by_one
    for gated in (False, True):
        p = problem(sgemm.IN_BF16, gated, 5, 3, 4, 33, 17, ids=torch.tensor([[0, 1, 2], [3, 3, -1], [4, 0, 0], [1, 2, 3], [9, -7, 1]]))
        for a, b in zip(reference(*p, gated), one_by_one(*p, gated)):
            assert float((a - b).abs().max()) <= 1e-12 * float(b.abs().max())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", [(1, 1, 1, 64, 64), (8, 2, 4, 128, 192), (9, 2, 4, 128, 64), (64, 4, 8, 256, 96), (5, 3, 4, 65, 33), (12, 2, 3, 301, 77), (64, 2, 4, 48, 1000)])
def test_24_bits_of_hidden_values(h, gated, T, J, E, W, F):  # noqa: F811
    """FP32 rows keep theirs in 24 bits, and small sizes are held to that (a few of the other file's, where 16
    bits are allowed for)."""
    check(h, sgemm.IN_F32, gated, problem(sgemm.IN_F32, gated, T, J, E, W, F))


# groups of 8, 16 and 32 tokens; one to four segments of 1024 bytes, the last one cut
STREAMED = [(4, 2, 3, 2064, 1040), (12, 2, 4, 2064, 1040), (16, 1, 2, 1040, 2064), (48, 2, 16, 2048, 1408), (64, 2, 16, 4096, 1040), (64, 4, 8, 2064, 1040), (33, 4, 4, 1040, 2064)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", STREAMED)
def test_through_shared_memory(h, kind, gated, T, J, E, W, F):  # noqa: F811
    check(h, kind, gated, problem(kind, gated, T, J, E, W, F))


# sixteen chunks of width a warp; many experts of narrow rows, where one, two or four warps share an item
IN_PLACE = [(5, 2, 3, 2500, 1001), (12, 2, 3, 3001, 1501), (64, 4, 4, 2501, 1040), (16, 4, 32, 65, 1001), (40, 2, 8, 100, 1010), (64, 3, 24, 250, 1001)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", IN_PLACE)
def test_on_any_alignment(h, kind, gated, T, J, E, W, F):  # noqa: F811
    check(h, kind, gated, problem(kind, gated, T, J, E, W, F))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T", [3, 20])
def test_tokens_beside_a_32_byte_boundary(h, kind, T):  # noqa: F811
    """Weights on boundaries, the tokens' rows 16, 8 and 2 or 4 bytes off, or apart by that much more."""
    p = problem(kind, True, T, 2, 4, 1040, 272)
    x, rest = p[0], [t.cuda() for t in p[1:]]
    want, err = reference(*p, True)
    size = x.element_size()
    for off, pad in ((16 // size, 0), (8 // size, 0), (1, 0), (0, 16 // size), (0, 1), (16 // size, 16 // size)):
        X = torch.full((off + T * (1040 + pad) + 64,), 99.0, dtype=x.dtype)
        X[off:off + T * (1040 + pad)].view(T, 1040 + pad)[:, :1040] = x
        X, out = X.cuda(), torch.full((T, 1040), 7.0, dtype=x.dtype, device="cuda")
        assert X.data_ptr() % 32 == 0
        ids, weights, up, us, down, ds = rest
        sgemm.sgemm_expert_layer_int8(h, kind, 1, T, 2, 4, 1040, 272, X[off:], 1040 + pad, ids, weights, up, us, down, ds, out, 1040)
        compare(out.cpu(), want, err)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("W,F", [(1040, 272), (1041, 270)])
@pytest.mark.parametrize("T,J,E", [(8, 2, 3), (20, 2, 3), (64, 4, 8)])
def test_infinities_and_nan_stay_in_their_token(h, kind, W, F, T, J, E):  # noqa: F811
    """A token with an infinity, one with a NaN, one with a NaN among its weights and one with a NaN for a choice
    that is left out: the others' results are as near to the 64-bit form as ever."""
    p = problem(kind, True, T, J, E, W, F)
    x, ids, weights, *rest = (t.clone() for t in p)
    x[1, 7], x[3, W - 1], weights[4, 0] = float("inf"), float("nan"), float("nan")
    ids[6, 1], weights[6, 1] = -1, float("nan")
    got = run(h, kind, True, (x, ids, weights, *rest))
    assert got[3].isnan().all() and got[4].isnan().all() and not got[1].isfinite().any()
    want, err = reference(x, ids, weights, *rest, True)
    compare(got, want, err, [t for t in range(T) if t not in (1, 3, 4)])


@pytest.mark.parametrize("T", [2, 24])
@pytest.mark.parametrize("W,F", [(1040, 272), (1041, 271)])
def test_weights_scales_and_choices_from_the_kernel_right_before(h, T, W, F):  # noqa: F811
    """The second kernel reads the routing, its weights and their scales before the first has ended, which began
    before the call's predecessor had: here the predecessors write them."""
    J, E, n = 2, 3, 4
    gen = torch.Generator(device="cuda").manual_seed(T + W)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ups, downs = ([randn(E * r, c).bfloat16() for _ in range(n)] for r, c in ((2 * F, W), (W, F)))
    chosen = [torch.randint(-1, E, (T, J), generator=gen, device="cuda", dtype=torch.int32) for _ in range(n)]
    shares = [torch.rand(T, J, generator=gen, device="cuda") for _ in range(n)]
    x = randn(T, W).bfloat16()
    up, us = torch.zeros(E, 2 * F, W, dtype=torch.int8, device="cuda"), torch.zeros(E, 2 * F, device="cuda")
    down, ds = torch.zeros(E, W, F, dtype=torch.int8, device="cuda"), torch.zeros(E, W, device="cuda")
    ids, weights = torch.zeros(T, J, dtype=torch.int32, device="cuda"), torch.zeros(T, J, device="cuda")

    def writers(i):
        yield lambda: sgemm.sgemm_quantize_rows(h, sgemm.IN_BF16, E * 2 * F, W, ups[i], W, up, W, us)
        yield lambda: sgemm.sgemm_quantize_rows(h, sgemm.IN_BF16, E * W, F, downs[i], F, down, F, ds)
        yield lambda: ids.copy_(chosen[i])
        yield lambda: weights.copy_(shares[i])

    def step(i, last, wait):
        out = torch.zeros_like(x)
        order = list(writers(i))
        for write in order[last + 1:] + order[:last + 1]:  # writer `last` comes right before the call
            write()
            if wait:
                torch.cuda.synchronize()
        sgemm.sgemm_expert_layer_int8(h, sgemm.IN_BF16, 1, T, J, E, W, F, x, W, ids, weights, up, us, down, ds, out, W)
        if wait:
            torch.cuda.synchronize()
        return out

    for last in range(4):
        want = [step(i, last, True) for i in range(n)]
        assert not torch.equal(want[0], want[1])
        for _ in range(3):
            got = [step(i, last, False) for i in range(n)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
