"""A pinned variant of the 4-bit products is the one that runs, whatever the sizes."""
import pytest

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_fp4 import FORMATS, check
from tests.test_gpu_fp4 import h, tile  # noqa: F401  (the handle; its reset)

pytestmark = pytest.mark.gpu

# (M, N, K), and what is chosen for it: few tokens, tiles of 128, pairs
SIZES = [((5, 300, 2500), sgemm.VARIANT_TC_F4), ((130, 260, 300), sgemm.VARIANT_TC_F4), ((2100, 2300, 400), sgemm.VARIANT_TC_F4_PAIR)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size,chosen", SIZES)
def test_pinned(h, tile, fmt, size, chosen):  # noqa: F811
    check(h, fmt, *size)
    assert sgemm.sgemm_last_variant(h)[0] == chosen
    for variant in (sgemm.VARIANT_TC_F4, sgemm.VARIANT_TC_F4_PAIR, sgemm.VARIANT_GENERIC_F4):
        sgemm.sgemm_set_variant(h, variant)
        check(h, fmt, *size)
        assert sgemm.sgemm_last_variant(h)[0] == variant
    sgemm.sgemm_set_variant(h, sgemm.VARIANT_AUTO)
    check(h, fmt, *size)
    assert sgemm.sgemm_last_variant(h)[0] == chosen
