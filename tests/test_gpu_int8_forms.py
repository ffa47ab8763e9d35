"""Further forms of the int8 products: what must hold whichever kernel, tile or
split runs.  Tolerances as in test_gpu_int8.py; kernels are compared bit for bit."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import FILL, Experts, handle, pinned  # noqa: F401  (fixtures)

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
