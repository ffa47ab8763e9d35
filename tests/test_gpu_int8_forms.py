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
