"""The tensor methods of the int8 and expert calls on a stream that is not the
current one: results come out right whatever is pending on the current stream,
and the memory that a pending call reads or writes is not given to others.

A stream is delayed by a kernel that spins for a fixed number of cycles; what the
results must equal is what the same calls give on the current stream."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm

pytestmark = pytest.mark.gpu

DELAY = 400_000_000      # cycles: 200 ms and more
T, J, E, W, N = 96, 2, 6, 512, 256


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    with sgemm.Sgemm() as handle:
        yield handle
        assert handle.device_status() == sgemm.OK


def inputs(g):
    gen = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def int8(*shape):
        return torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)

    ids = torch.randint(0, E, (T, J), generator=gen, device="cuda", dtype=torch.int32)
    ids[::5, 0] = -1                                   # rows that no slot has
    offsets, rows, _ = g.expert_sort(ids, E)
    return dict(ids=ids, offsets=offsets, rows=rows, x=randn(T, W).bfloat16(), y=randn(T * J, W).bfloat16(),
                dout=randn(T, W).bfloat16(), weights=torch.rand(T, J, generator=gen, device="cuda"), a=int8(T * J, W),
                sa=torch.rand(T * J, generator=gen, device="cuda"), b=int8(E, N, W),
                sb=torch.rand(E, N, generator=gen, device="cuda"))


METHODS = {
    "quantize": lambda g, d, s: g.quantize(d["x"], stream=s),
    "matmul_int8": lambda g, d, s: g.matmul_int8(d["a"], d["sa"], d["b"][0], d["sb"][0], stream=s),
    "matmul_int8_experts": lambda g, d, s: g.matmul_int8_experts(d["offsets"], d["a"], d["sa"], d["b"], d["sb"], stream=s),
    "expert_sort": lambda g, d, s: g.expert_sort(d["ids"], E, stream=s),
    "expert_dispatch": lambda g, d, s: g.expert_dispatch(d["x"], d["rows"], stream=s),
    "expert_dispatch_int8": lambda g, d, s: g.expert_dispatch_int8(d["x"], d["rows"], stream=s),
    "expert_dispatch_grad": lambda g, d, s: g.expert_dispatch_grad(d["y"], d["rows"], stream=s),
    "expert_combine": lambda g, d, s: g.expert_combine(d["y"], d["rows"], d["weights"], stream=s),
    "expert_combine_grad": lambda g, d, s: g.expert_combine_grad(d["dout"], d["y"], d["rows"], d["weights"], stream=s),
}


def tensors(result):
    return result if isinstance(result, tuple) else (result,)


def prepare(g, name):
    """(inputs, expected results, another stream), everything loaded that the first
    use of a kernel or of a stream's pool loads (which may wait for the GPU)."""
    d = inputs(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    METHODS[name](g, d, side)
    want = [t.clone() for t in tensors(METHODS[name](g, d, None))]
    for t in (torch.empty_like(t) for t in (*want, *d.values())):
        t.fill_(77)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    return d, want, side


@pytest.mark.parametrize("name", list(METHODS))
@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_results_do_not_wait_for_or_mix_with_the_current_stream(g, name, as_handle):
    """The current stream spins, then overwrites memory of the results' sizes that it
    has given back: nothing of that may reach the results."""
    d, want, side = prepare(g, name)
    torch.cuda._sleep(DELAY)
    freed = [torch.empty_like(t) for t in want]
    for t in freed:
        t.fill_(77)
    del freed, t
    got = tensors(METHODS[name](g, d, side.cuda_stream if as_handle else side))
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was not busy any more: nothing was tested"
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", list(METHODS))
def test_inputs_stay_until_the_stream_has_read_them(g, name):
    """The side stream spins; meanwhile the inputs are dropped and the current stream
    fills new tensors of their sizes."""
    d, want, side = prepare(g, name)
    sizes = {k: (t.shape, t.dtype) for k, t in d.items()}
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = tensors(METHODS[name](g, d, side))
    d.clear()
    new = [torch.empty(shape, dtype=dtype, device="cuda").fill_(77) for shape, dtype in sizes.values()]
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the side stream had read its inputs: nothing was tested"
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del new


def test_the_default_stream_by_its_handle(g):
    d = inputs(g)
    want = g.expert_dispatch(d["x"], d["rows"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = g.expert_dispatch(d["x"], d["rows"], stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
