"""Norm, 4-bit and expert-layer calls of two handles on two streams at once, each with workspaces of its own:
the bits that each gives alone.  And an expert layer whose weights are past 2^31 bytes."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import build, sgemm
from tests.test_gpu_rows_together import FORMATS, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handles():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    with sgemm.Sgemm() as a, sgemm.Sgemm() as b:
        yield a, b
        torch.cuda.synchronize()
        assert a.device_status() == b.device_status() == sgemm.OK


def close(d, g, M, K):
    """A backward pass too, which adds up in the workspace."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    x, w, dy = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((M, K), (K,), (M, K)))
    _, _, rstd = g.rms_norm(x, w)
    torch.cuda.synchronize()
    return lambda: g.rms_norm_grad(dy, x, w, rstd)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("one,other", [((5, 256, 640), (700, 1000, 300)), ((300, 512, 512), (40, 330, 1001)), ((2100, 2300, 400), (12, 4096, 4096))])
def test_at_once(handles, fmt, one, other):
    steps = [Step(fmt, *one, 1), Step(fmt, *other, 2)]
    grads = [close(i, g, s.M, s.K) for i, (g, s) in enumerate(zip(handles, steps))]
    want = []
    for g, s, grad in zip(handles, steps, grads):
        want.append([*s.run(g.h, 6, wait=True), *grad()])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s in steps:
            s.residual.zero_()
        torch.cuda.synchronize()
        kept = [[], []]
        for i in range(6):
            todo = [list(s.calls(g.h, i)) for g, s in zip(handles, steps)]
            for calls in zip(*todo):        # the two streams' calls in turn
                for call, stream in zip(calls, streams):
                    with torch.cuda.stream(stream):
                        call()
            for n, (s, stream) in enumerate(zip(steps, streams)):
                with torch.cuda.stream(stream):
                    kept[n] += [s.y.clone(), s.z.clone(), s.out.clone(), s.residual.clone()]
        for n, (grad, stream) in enumerate(zip(grads, streams)):
            with torch.cuda.stream(stream):
                kept[n] += grad()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("W,F", [(16384, 8192), (16383, 8193)])
def test_layer_with_weights_past_2_31_bytes(handles, W, F):
    """The last experts' tokens: the bits of a layer that has these alone."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("too little free memory")
    g, E, T = handles[0], 19, 3
    gen = torch.Generator(device="cuda").manual_seed(W)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=gen, dtype=torch.int8, device="cuda")  # noqa: E731
    up, down = i8(E, F, W), i8(E, W, F)
    assert up[:-2].numel() > 1 << 31 and down[:-2].numel() > 1 << 31
    us, ds = torch.rand(E, F, generator=gen, device="cuda") / 9999, torch.rand(E, W, generator=gen, device="cuda") / 9999
    x, weights = torch.randn(T, W, generator=gen, device="cuda").bfloat16(), torch.rand(T, 2, generator=gen, device="cuda")
    ids = torch.tensor([[0, 1], [1, -1], [1, 0]], dtype=torch.int32, device="cuda")
    got = g.expert_layer_int8(x, torch.where(ids >= 0, ids + E - 2, ids), weights, up, us, down, ds)
    want = g.expert_layer_int8(x, ids, weights, up[-2:].clone(), us[-2:].clone(), down[-2:].clone(), ds[-2:].clone())
    assert torch.equal(got, want) and bool((got != 0).any(dim=1).all())
