"""What the getters report after the quantization and routing calls: the last
successful call's launches, also where a later call was refused."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_experts import CALLS

pytestmark = pytest.mark.gpu

V = sgemm


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


def report(h):
    return (*sgemm.sgemm_last_variant(h), sgemm.sgemm_last_launches(h), sgemm.sgemm_last_relayout(h))


def after_a_product(h):
    """The report of an FP32 product, which no quantization or routing call leaves."""
    a = torch.zeros(64, 64, device="cuda")
    sgemm.sgemm_run(h, 64, 64, 64, 1.0, a, 64, a, 64, 0.0, torch.zeros(64, 64, device="cuda"), 64)
    got = report(h)
    assert got[0] >= 0 and got[2] >= 1
    return got


def call_of(name):
    if name == "quantize":
        return sgemm.sgemm_quantize_rows, dict(in_type=V.IN_F32, M=3, K=16), ["X", "ldx", "Q", "ldq", "scale"], "M"
    if name == "sort":
        return sgemm.sgemm_expert_sort, dict(tokens=3, choices=2, experts=4), ["ids", "offsets", "rows", "source"], "tokens"
    call, names, _ = CALLS[name]
    return call, dict(in_type=V.IN_F32, tokens=3, choices=2, width=16), names, "tokens"


@pytest.mark.parametrize("name", ["quantize", "sort", *CALLS])
def test_a_refused_call_changes_no_report(handle, name):
    call, args, names, count = call_of(name)
    ints = ("rows", "ids", "offsets", "source")
    bufs = {n: torch.zeros(256, dtype=torch.int8 if n == "Q" else torch.int32 if n in ints else torch.float32,
                           device="cuda") for n in names if not n.startswith("ld")}
    args = {**args, **{n: 16 if n.startswith("ld") else bufs[n] for n in names}}
    before = after_a_product(handle)
    first, second = list(bufs)[0], list(bufs)[-1]
    for bad in (dict([(first, None)]), dict([(second, None)]), dict([(second, bufs[second].data_ptr() + 1)]),
                dict([(second, bufs[first])]), dict([(count, -1)])):
        with pytest.raises(sgemm.SgemmError):
            call(handle, **{**args, **bad})
        assert report(handle) == before, bad
    call(handle, **args)
    assert report(handle) == (-1, 1, 1, 0)
    after_a_product(handle)
    call(handle, **{**args, count: 0})
    assert report(handle) == (-1, 1, 1 if name == "sort" else 0, 0)   # (the sort writes offsets of no slots)
    torch.cuda.synchronize()
