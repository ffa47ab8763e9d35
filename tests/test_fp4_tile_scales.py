"""Plain scales laid out in tiles: the sizes without a row or an element, and what is refused.  No GPU."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return sgemm.lib()


@pytest.mark.parametrize("fmt", [sgemm.FP4_MX, sgemm.FP4_NV])
@pytest.mark.parametrize("rows,K", [(0, 0), (0, 64), (0, 7), (3, 0), (200, 0)])
def test_nothing_to_lay_out(fmt, rows, K):
    """The calls take rows of no elements, and no rows: their scales are as many bytes as the library says, none."""
    t = sgemm.fp4_tile_scales(torch.zeros(rows, sgemm.fp4_blocks(fmt, K), dtype=torch.uint8), fmt, K)
    assert t.dtype == torch.uint8 and t.shape == (sgemm.sgemm_fp4_scale_bytes(fmt, rows, K),) == (0,)


@pytest.mark.parametrize("fmt", [2, -1])
def test_unknown_formats_are_refused(fmt):
    with pytest.raises(ValueError, match="format"):
        sgemm.fp4_blocks(fmt, 32)
    for blocks in (1, 2):
        with pytest.raises(ValueError, match="format"):
            sgemm.fp4_tile_scales(torch.zeros(4, blocks, dtype=torch.uint8), fmt, 32)
