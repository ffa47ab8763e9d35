"""Stream order of the quantization, int8 and routing calls: each launch may begin
while the kernel before it ends, so what one call writes the next one has to read
fresh, in the same buffers again and again, by every kind of load -- none of it
may come from what a cache of the SM held of the buffer's contents before.

Both operands of a product are quantized anew before each of them, with no
synchronisation in between; results equal those of the same calls with one after
each."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from tests.test_gpu_int8 import handle, pinned  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

V = sgemm
STEPS = 24


@pytest.mark.parametrize("variant,M,N,K,trans_b", [
    (V.VARIANT_FEW_I8, 8, 333, 1001, 1), (V.VARIANT_FEW_I8, 1, 2000, 1024, 1), (V.VARIANT_GENERIC_I8, 70, 333, 1001, 1),
    (V.VARIANT_GENERIC_I8, 70, 1001, 333, 0), (V.VARIANT_TC_I8, 40, 333, 1001, 1), (V.VARIANT_TC_I8, 40, 1001, 333, 0),
    (V.VARIANT_TC_I8, 40, 512, 1024, 1), (V.VARIANT_TC_I8, 700, 1000, 1001, 0), (V.VARIANT_TC_I8, 700, 4096, 1024, 1)])
def test_operands_written_by_the_call_before(handle, pinned, variant, M, N, K, trans_b):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    rows, cols = (N, K) if trans_b else (K, N)
    X = torch.randn(3, M, K, generator=g, device="cuda")
    W = torch.randn(3, rows, cols, generator=g, device="cuda")
    a, b = (torch.empty(r, c, dtype=torch.int8, device="cuda") for r, c in ((M, K), (rows, cols)))
    sa, sw = torch.empty(M, device="cuda"), torch.empty(rows, device="cuda")
    sb = torch.rand(N, generator=g, device="cuda")
    pinned(variant)

    def step(i, C, wait):
        for call in (lambda: sgemm.sgemm_quantize_rows(handle, V.IN_F32, rows, cols, W[i % 3], cols, b, cols, sw),
                     lambda: sgemm.sgemm_quantize_rows(handle, V.IN_F32, M, K, X[i % 2], K, a, K, sa),
                     lambda: sgemm.sgemm_run_int8(handle, trans_b, V.IN_F32, M, N, K, a, K, sa, b, cols, sb, None, C, N)):
            call()
            if wait:
                torch.cuda.synchronize()

    want, got = (torch.empty(STEPS, M, N, device="cuda") for _ in range(2))
    for i in range(STEPS):
        step(i, want[i], True)
    for i in range(STEPS):
        step(i, got[i], False)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("tokens,choices,width", [(40, 2, 256), (3000, 2, 640), (3000, 4, 2048)])
def test_routes_written_by_the_call_before(handle, tokens, choices, width):  # noqa: F811
    experts, slots = 16, tokens * choices
    g = torch.Generator(device="cuda").manual_seed(tokens + width)
    ids = torch.randint(0, experts, (3, tokens, choices), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(tokens, width, generator=g, device="cuda")
    dout = torch.randn(tokens, width, generator=g, device="cuda")
    weights = torch.rand(tokens, choices, generator=g, device="cuda")
    off, rows, source = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts + 1, slots, slots))
    y, dy = (torch.zeros(slots, width, device="cuda") for _ in range(2))

    def step(i, out, dw, dx, wait):
        for call in (lambda: sgemm.sgemm_expert_sort(handle, tokens, choices, experts, ids[i % 3], off, rows, source),
                     lambda: sgemm.sgemm_expert_dispatch(handle, V.IN_F32, tokens, choices, width, x, width, rows, y, width),
                     lambda: sgemm.sgemm_expert_combine(handle, V.IN_F32, tokens, choices, width, y, width, rows, weights, out,
                                                        width),
                     lambda: sgemm.sgemm_expert_combine_grad(handle, V.IN_F32, tokens, choices, width, dout, width, y, width,
                                                             rows, weights, dy, width, dw),
                     lambda: sgemm.sgemm_expert_dispatch_grad(handle, V.IN_F32, tokens, choices, width, dy, width, rows, dx,
                                                              width)):
            call()
            if wait:
                torch.cuda.synchronize()

    results = [[torch.empty(STEPS, *shape, device="cuda") for shape in ((tokens, width), (tokens, choices), (tokens, width))]
               for _ in range(2)]
    for wait, r in zip((True, False), results):
        for i in range(STEPS):
            step(i, r[0][i], r[1][i], r[2][i], wait)
        torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)
