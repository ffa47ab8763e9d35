"""Further forms of the int8 products: what must hold whichever kernel, tile or
split runs.  Tolerances as in test_gpu_int8.py; kernels are compared bit for bit."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import FILL, Experts, Problem, handle, pinned  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

V = sgemm


def in_order(offsets, rows):
    """The nearest bounds that are in order: each offset kept within [0, rows] and not below the ones before."""
    out, top = [], 0
    for x in offsets:
        top = max(top, min(max(x, 0), rows))
        out.append(top)
    return torch.tensor(out, dtype=torch.int32)


@pytest.mark.parametrize("bad", [[0, 50, 20, 30], [-5, 10, 999, 40], [40, 30, 20, 10], [999, 999, 999, 999], [0, 30, 10, 20],
                                 [5, 25, 12, 40], [0, 0, -1, 40], [0, 10, 20, 5]])
@pytest.mark.parametrize("variant", [V.VARIANT_TC_I8, V.VARIANT_GENERIC_I8])
def test_offsets_out_of_order_are_the_nearest_in_order(handle, pinned, bad, variant):  # noqa: F811
    """Every row is the product with the expert that owns it then; rows of none keep what they held."""
    p = Experts([10, 20, 10], 64, 64, "f32", bias=True, seed=6)
    pinned(variant)
    got = p.run(handle, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert sgemm.sgemm_last_variant(handle)[0] == variant
    p.offsets = in_order(bad, p.R)
    p.check(got)
    assert bool((got[p.R] == FILL).all())


@pytest.mark.parametrize("variant", [V.VARIANT_TC_I8, V.VARIANT_GENERIC_I8])
def test_many_offsets_out_of_order(handle, pinned, variant):  # noqa: F811
    """More offsets than a block has threads, their running maximum set by one far back."""
    E = 700
    p = Experts([1] * E, 40, 48, "f32", seed=7)
    offsets = torch.arange(E + 1, dtype=torch.int32)
    offsets[3] = 400                                    # experts 3 .. 399 own nothing, expert 2 owns 398 rows
    offsets[650] = 0
    pinned(variant)
    got = p.run(handle, offsets.cuda())
    p.offsets = in_order(offsets.tolist(), p.R)
    p.check(got)


@pytest.mark.parametrize("M,N,K,variant", [(1, 300, 1001, V.VARIANT_FEW_I8), (8, 700, 701, V.VARIANT_FEW_I8),
                                           (8, 4096, 4097, V.VARIANT_FEW_I8), (3, 9000, 301, V.VARIANT_FEW_I8),
                                           (8, 9000, 33, V.VARIANT_GENERIC_I8), (9, 300, 1001, V.VARIANT_GENERIC_I8)])
def test_few_tokens_where_b_may_not_be_copied(handle, pinned, M, N, K, variant):  # noqa: F811
    """Without the copy the tensor cores cannot run: the kernel for few tokens, which
    reads B in place, is weighed against the generic one and not against them."""
    p = Problem(M, N, K, "bf16", bias=True, seed=9)
    sgemm.sgemm_set_relayout(handle, V.RELAYOUT_OFF)
    first = p.run(handle)
    assert sgemm.sgemm_last_variant(handle)[0] == variant
    p.check(first)
    pinned(V.VARIANT_GENERIC_I8)
    assert torch.equal(p.run(handle), first)


# ---- B stored K x N past 2^31 elements ---------------------------------------------
@pytest.mark.parametrize("variant", [V.VARIANT_TC_I8, V.VARIANT_GENERIC_I8])
@pytest.mark.parametrize("off", [0, 1])
def test_a_k_by_n_matrix_with_far_rows(handle, pinned, variant, off):  # noqa: F811
    """Rows of B 2^19 bytes apart, the last ones past 2^31: copied, or read in place."""
    M, N, K, ldb = 20, 72, 4200, (1 << 19) + off
    g = torch.Generator(device="cuda").manual_seed(40)
    B = torch.randint(-127, 128, ((K - 1) * ldb + N,), dtype=torch.int8, device="cuda", generator=g)
    b = B.as_strided((K, N), (ldb, 1)).double()
    A = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sb, C = torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.zeros(M, N, device="cuda")
    pinned(variant)
    sgemm.sgemm_run_int8(handle, 0, V.IN_F32, M, N, K, A, K, sa, B, ldb, sb, None, C, N)
    torch.cuda.synchronize()
    assert sgemm.sgemm_last_variant(handle)[0] == variant
    assert sgemm.sgemm_last_relayout(handle) == (2 if variant == V.VARIANT_TC_I8 else 0)
    assert torch.equal(C, (A.double() @ b).float())


@pytest.mark.parametrize("variant", [V.VARIANT_TC_I8, V.VARIANT_GENERIC_I8])
def test_far_experts_with_k_by_n_matrices(handle, pinned, variant):  # noqa: F811
    """Experts' matrices 2^28 bytes apart: copied a small piece of each, or read in place."""
    E, N, K, stride, rows = 10, 130, 200, 1 << 28, 40
    g = torch.Generator(device="cuda").manual_seed(41)
    B = torch.randint(-127, 128, ((E - 1) * stride + K * N,), dtype=torch.int8, device="cuda", generator=g)
    A = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    offsets = torch.tensor([0, 3, 3, 10, 11, 11, 11, 20, 20, 25, 40], dtype=torch.int32, device="cuda")
    sa, sb = torch.ones(rows, device="cuda"), torch.ones(E, N, device="cuda")
    C = torch.zeros(rows, N, device="cuda")
    pinned(variant)
    sgemm.sgemm_run_int8_experts(handle, 0, V.IN_F32, E, rows, N, K, offsets, A, K, sa, B, N, stride, sb, None, C, N)
    torch.cuda.synchronize()
    assert sgemm.sgemm_last_variant(handle)[0] == variant
    at = offsets.tolist()
    for e in range(E):
        b = B[e * stride:e * stride + K * N].view(K, N).double()
        assert torch.equal(C[at[e]:at[e + 1]], (A[at[e]:at[e + 1]].double() @ b).float())


def test_experts_beyond_the_workspace(handle):  # noqa: F811
    """K x N matrices whose copies do not fit: the generic kernel, offsets past 2^31."""
    E, N, K, rows = 9, 1 << 15, 8192, 6
    g = torch.Generator(device="cuda").manual_seed(42)
    B = torch.randint(-127, 128, (E, K, N), dtype=torch.int8, device="cuda", generator=g)
    A = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    offsets = torch.tensor([0] * (E - 1) + [2, rows], dtype=torch.int32, device="cuda")
    sa, sb = torch.ones(rows, device="cuda"), torch.ones(E, N, device="cuda")
    C = torch.zeros(rows, N, device="cuda")
    sgemm.sgemm_run_int8_experts(handle, 0, V.IN_F32, E, rows, N, K, offsets, A, K, sa, B, N, N * K, sb, None, C, N)
    torch.cuda.synchronize()
    assert sgemm.sgemm_last_variant(handle)[0] == V.VARIANT_GENERIC_I8
    at = torch.tensor([0, 1, 777, N - 2, N - 1], device="cuda")
    for e, lo, hi in [(E - 2, 0, 2), (E - 1, 2, rows)]:
        assert torch.equal(C[lo:hi, at], (A[lo:hi].double() @ B[e][:, at].double()).float())
