"""The whole expert layer on FP32 rows, as near to the 64-bit form as sums of FP32 products come.

A tensor core's sum is truncated, by up to 2^-23 of itself an MMA and always towards zero, so that a chain of
MMAs drifts by as many: 64 terms of a sum are four MMAs (their low parts, 2^-8 of them and less, are
added first), and what these give is added up with rounding to nearest.  Over the whole result, in which
the errors of single elements average: 4 steps of 2^-23 for each of the three sums (gate, factor, second
product), and 4 for what is rounded besides (silu, scales, products, the sums of chunks and warps)."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_expert_layer_few import problem, run
from tests.test_gpu_expert_layer_wide import reference
from tests.test_gpu_expert_layer_few import h  # noqa: F401  (the handle)

pytestmark = pytest.mark.gpu

SIZES = [(27, 1, 32, 72, 1159), (2, 2, 8, 644, 1544), (1, 2, 8, 3705, 613), (2, 2, 16, 4085, 181), (12, 2, 4, 749, 353), (40, 2, 4, 2001, 1001),  # any alignment
         (1, 2, 4, 4096, 2064), (8, 2, 4, 2064, 1040), (12, 2, 4, 1040, 2064), (48, 2, 4, 2048, 1408), (64, 2, 2, 4096, 1040)]               # through shared memory


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,J,E,W,F", SIZES)
def test_error_on_the_whole(h, gated, T, J, E, W, F):  # noqa: F811
    p = problem(sgemm.IN_F32, gated, T, J, E, W, F, seed=7)
    got = run(h, sgemm.IN_F32, gated, p).double()
    want, _ = reference(*p, gated)
    assert float((got - want).norm()) <= 16 * 2.0 ** -23 * float(want.norm())
