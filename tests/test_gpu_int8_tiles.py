"""Every token tile and K split of the int8 products on the tensor cores, each
held by the test hook: the sum is an exact integer whatever the tile, so the bits
of the generic kernel are the bits of all of them; the generic kernel's and one
form's own results are held against 64 bits elsewhere and here."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import FILL, TYPES, Experts, Problem, handle  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

V = sgemm
DIRECT = [(t, s) for t in (16, 32, 64) for s in (1, 2, 4, 8)]
PAIRS = [(128, 1), (256, 1)]
TILES = DIRECT + PAIRS
NAMES = [f"{t}x{s}" for t, s in TILES]


@pytest.fixture
def tile(handle):  # noqa: F811
    """tile(t, s): later products on the tensor cores take this tile and split.  generic(): on the generic kernel."""
    def hold(tokens, ksplit):
        sgemm.sgemm_set_variant(handle, V.VARIANT_TC_I8)
        sgemm.sgemm_debug_set_int8_tile(handle, tokens, ksplit)
    yield hold
    sgemm.sgemm_debug_set_int8_tile(handle, 0, 0)
    sgemm.sgemm_set_variant(handle, V.VARIANT_AUTO)


def same_as_generic(h, p, got):
    sgemm.sgemm_set_variant(h, V.VARIANT_GENERIC_I8)
    p.C.fill_(FILL)
    want = p.run(h)
    assert sgemm.sgemm_last_variant(h)[0] == V.VARIANT_GENERIC_I8
    word = torch.int32 if got.dtype == torch.float32 else torch.int16
    assert torch.equal(got.view(word), want.view(word))


def stages(K):
    return (K + 127) // 128


def ran(h, tokens, ksplit, K):
    variant, splits = sgemm.sgemm_last_variant(h)
    while ksplit > stages(K):
        ksplit //= 2
    assert (variant, splits) == (V.VARIANT_TC_I8, ksplit)
    if tokens > 64:
        assert sgemm.sgemm_last_launches(h) >= 2        # the tokens' conversion, and the product


def test_the_hook_refuses_what_is_no_tile(handle):  # noqa: F811
    for tokens, ksplit in TILES + [(0, 0)]:
        sgemm.sgemm_debug_set_int8_tile(handle, tokens, ksplit)
    for tokens, ksplit in [(0, 1), (8, 1), (16, 0), (16, 3), (16, 16), (48, 1), (128, 0), (128, 2), (256, 2), (512, 1),
                           (-16, 1), (16, -1)]:
        with pytest.raises(sgemm.SgemmError):
            sgemm.sgemm_debug_set_int8_tile(handle, tokens, ksplit)


# channels on both sides of 128 and 256; one stage of k, odd and even numbers of
# them, whole and not; tokens around a tile's half and end, one tile and several
SIZES = [(1, 1), (129, 40), (256, 128), (257, 300), (300, 1024), (130, 1153), (384, 4100)]


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_parity(handle, tile, tokens, ksplit, N, K, dtype):  # noqa: F811
    T = tokens
    for i, M in enumerate([1, T // 2 - 1, T // 2, T // 2 + 1, T - 1, T, T + 1, T + T // 2, 2 * T + 3]):
        p = Problem(M, N, K, dtype, bias=i % 2 == 0, pads=(0, 0, i % 3), seed=20 + i)
        tile(tokens, ksplit)
        got = p.run(handle)
        ran(handle, tokens, ksplit, K)
        p.check(got)
        same_as_generic(handle, p, got)


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
@pytest.mark.parametrize("trans_b,pads,offsets", [(1, (16, 32, 2), (32, 16, 2)), (1, (1, 7, 1), (3, 5, 1)),
                                                  (0, (0, 0, 0), (0, 0, 0)), (0, (5, 3, 0), (1, 2, 3))])
def test_layouts(handle, tile, tokens, ksplit, trans_b, pads, offsets):  # noqa: F811
    p = Problem(tokens + 5, 270, 1000, "bf16", trans_b=trans_b, bias=True, pads=pads, offsets=offsets, seed=30)
    tile(tokens, ksplit)
    got = p.run(handle)
    ran(handle, tokens, ksplit, 1000)
    p.check(got)
    same_as_generic(handle, p, got)


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
def test_more_tiles_than_places(handle, tile, tokens, ksplit):  # noqa: F811
    """A CTA (cluster, pair) works through several tiles, an uneven number of them."""
    tiles = 2 * 170 if tokens > 64 else 2 * 340
    p = Problem(tokens * tiles // 4 + 7, 4 * (256 if tokens > 64 else 128) - 30, 900, "f16", bias=True, seed=31)
    tile(tokens, ksplit)
    got = p.run(handle)
    ran(handle, tokens, ksplit, 900)
    p.check(got)
    same_as_generic(handle, p, got)


# ---- sums at the ends of what the accumulators hold --------------------------------
def exact_sums(h, M, N, K, fill_a, fill_b):
    """A product with scales of 1 into FP32: the integers themselves."""
    p = Problem(M, N, K, "f32", unit=True, seed=32)
    fill_a(p.a)
    fill_b(p.b)
    p.A.copy_(p.a)
    p.B.copy_(p.b)
    got = p.run(h)
    want = (p.a.double().cuda() @ p.b.double().cuda().t()).cpu().float()
    assert torch.equal(got, want)


def const(v, step=0, other=0):
    def fill(x):
        x.fill_(v)
        if step:
            x[:, ::step] = other
    return fill


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
@pytest.mark.parametrize("fill_a,fill_b", [
    (const(-128), const(-128)),                 # the largest products: 1024 of them are 2^24
    (const(127), const(127)),
    (const(127, 3, 125), const(127, 5, 121)),   # odd sums near 2^24
    (const(-128), const(127, 2, -127)),         # sums that stay small
], ids=["low", "high", "odd", "mixed"])
def test_extremes(handle, tile, tokens, ksplit, fill_a, fill_b):  # noqa: F811
    tile(tokens, ksplit)
    for K in (1024, 1152, 9000):
        exact_sums(handle, tokens + 9, 140, K, fill_a, fill_b)
        ran(handle, tokens, ksplit, K)


def chunk(top):
    """Stages of 128 k that the pair kernel lets run between two drains, where the
    largest sum of |a| over 512 k is `top`: c windows of 512 and one more hold it, and
    128 (c + 1) top <= 2^24."""
    return max(4 * ((1 << 17) // top - 1) & ~1, 8)


@pytest.mark.parametrize("tokens", [128, 256])
@pytest.mark.parametrize("value,other", [(1, 1), (1, -1), (16, 16), (15, 17), (3, 2), (60, 61)])
def test_long_runs_between_drains(handle, tile, tokens, value, other):  # noqa: F811
    """Small tokens against B of -128 and 127: K at one run's end, one stage and one k
    beyond, and several runs; all products of one sign, the longest sums there can be."""
    run = chunk(512 * max(abs(value), abs(other)))
    tile(tokens, 1)
    for K in sorted({min(k, 131071) for k in (run * 128 - 1, run * 128, run * 128 + 1, run * 128 + 129, run * 256 + 300)}):
        if K > 40000 and (value, other) not in ((1, 1), (1, -1)):
            continue
        for b in (const(-128), const(127, 7, 126)):
            exact_sums(handle, tokens // 2 + 3, 40, K, const(value, 2, other), b)
            ran(handle, tokens, 1, K)


@pytest.mark.parametrize("tokens", [128, 256])
@pytest.mark.parametrize("top", [2, 11, 40, 127])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_runs_of_other_sizes(handle, tile, tokens, top, dtype):  # noqa: F811
    """Random tokens of magnitude up to `top`, one row of zeros and one row larger than the others."""
    p = Problem(tokens + tokens // 2 + 1, 300, 6500, dtype, bias=True, seed=33)
    p.a.clamp_(-top, top)
    p.a[3] = 0
    p.a[tokens // 2] = min(2 * top, 127)
    p.A.copy_(p.a)
    tile(tokens, 1)
    got = p.run(handle)
    ran(handle, tokens, 1, 6500)
    p.check(got)
    same_as_generic(handle, p, got)


# ---- by expert ---------------------------------------------------------------------
def counts_for(T):
    """Groups whose last tile is up to half a tile, more, or whole; empty ones; single rows."""
    return [T + T // 4, T // 2, T // 2 + 1, 0, 1, 2 * T + 1, 2 * T + T // 2, T, 0, 3 * T - 1]


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
@pytest.mark.parametrize("N,K", [(200, 160), (257, 1153)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_experts(handle, tile, tokens, ksplit, N, K, dtype):  # noqa: F811
    p = Experts(counts_for(tokens), N, K, dtype, bias=K > 1000, before=3, after=9, seed=34)
    tile(tokens, ksplit)
    got = p.run(handle)
    ran(handle, tokens, ksplit, K)
    p.check(got)
    same_as_generic(handle, p, got)


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
@pytest.mark.parametrize("trans_b,pad,shared", [(0, 0, False), (1, 1, False), (1, 0, True)])
def test_experts_layouts(handle, tile, tokens, ksplit, trans_b, pad, shared):  # noqa: F811
    p = Experts(counts_for(tokens), 150, 272, "f32", trans_b=trans_b, pad=pad, shared=shared, bias=True, seed=35)
    tile(tokens, ksplit)
    got = p.run(handle)
    ran(handle, tokens, ksplit, 272)
    p.check(got)
    same_as_generic(handle, p, got)


@pytest.mark.parametrize("tokens,ksplit", TILES, ids=NAMES)
def test_one_expert_has_nearly_all_rows(handle, tile, tokens, ksplit):  # noqa: F811
    """Many experts, most of them with a row or none; more tiles than places."""
    counts = [i % 3 == 0 for i in range(60)] + [tokens * 90 + 5] + [i % 2 for i in range(70)]
    p = Experts([int(c) for c in counts], 520, 700, "bf16", seed=36)
    tile(tokens, ksplit)
    got = p.run(handle)
    ran(handle, tokens, ksplit, 700)
    p.check(got)
    same_as_generic(handle, p, got)


@pytest.mark.parametrize("tokens", [128, 256])
def test_a_pass_that_starts_inside_an_expert(handle, tile, tokens):  # noqa: F811
    """The tokens' FP16 rows of 32 KiB fill the workspace after 16384 of them, less what
    stands before: the second pass starts inside the second expert."""
    g = torch.Generator(device="cuda").manual_seed(37)
    counts, N, K = [9000, 7900, 1, 300], 200, 16384
    R = sum(counts) + 5
    offsets = torch.tensor([0, 9000, 16900, 16901, 17201], dtype=torch.int32, device="cuda")
    A = torch.randint(-128, 128, (R, K), dtype=torch.int8, device="cuda", generator=g)
    B = torch.randint(-128, 128, (4, N, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(R, device="cuda", generator=g), torch.rand(4, N, device="cuda", generator=g)
    bias = torch.randn(4, N, device="cuda", generator=g)
    results = []
    for t in (tokens, 0):
        C = torch.full((R, N), FILL, device="cuda")
        tile(t, 1) if t else sgemm.sgemm_set_variant(handle, V.VARIANT_GENERIC_I8)
        sgemm.sgemm_run_int8_experts(handle, 1, V.IN_F32, 4, R, N, K, offsets, A, K, sa, B, K, N * K, sb, bias, C, N)
        torch.cuda.synchronize()
        if t:
            assert sgemm.sgemm_last_launches(handle) == 4
        results.append(C)
    assert torch.equal(*results)
    assert bool((results[0][17201:] == FILL).all())
    for r, e in [(0, 0), (8999, 0), (9000, 1), (16383, 1), (16384, 1), (16899, 1), (16900, 2), (17200, 3)]:
        prod = (A[r].double() @ B[e].double().t()) * sb[e].double() * sa[r].double()
        want = prod + bias[e].double()
        assert bool(((results[0][r].double() - want).abs() <= 3.1 * 2.0 ** -24 * prod.abs() + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("tokens,ksplit", [(16, 4), (64, 1)])
def test_passes_over_realigned_rows(handle, tile, tokens, ksplit):  # noqa: F811
    """The same for rows that are copied onto 16-byte boundaries."""
    g = torch.Generator(device="cuda").manual_seed(38)
    M, N, K = 9000, 40, 65537
    A = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    B = torch.randint(-128, 128, (N, K + 15), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    C = torch.zeros(M, N, device="cuda")
    tile(tokens, ksplit)
    sgemm.sgemm_run_int8(handle, 1, V.IN_F32, M, N, K, A, K, sa, B, K + 15, sb, None, C, N)
    torch.cuda.synchronize()
    assert sgemm.sgemm_last_launches(handle) == 4 and sgemm.sgemm_last_variant(handle) == (V.VARIANT_TC_I8, ksplit)
    b = B[:, :K].double().t()
    for r in range(0, M, 1500):
        assert torch.equal(C[r:r + 1500], (A[r:r + 1500].double() @ b).float())


def test_the_tiles_that_are_chosen(handle):  # noqa: F811
    """Without the hook, on shapes that the choice gives to each kernel: the same bits."""
    sgemm.sgemm_set_variant(handle, V.VARIANT_AUTO)
    for M, N, K, launches in [(40, 4096, 4096, 1), (256, 4096, 4096, 1), (512, 4096, 2048, 2), (2048, 2048, 1024, 2)]:
        p = Problem(M, N, K, "bf16", seed=39)
        got = p.run(handle)
        assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_TC_I8
        assert sgemm.sgemm_last_launches(handle) == launches, (M, N, K)
        p.check(got)
        same_as_generic(handle, p, got)
        sgemm.sgemm_set_variant(handle, V.VARIANT_AUTO)
