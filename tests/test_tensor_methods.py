"""What the tensor methods of the int8 and expert calls refuse before they reach
the library.  No GPU: tensors that the kernels could not address never get there."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm

T, J, E, W, N = 4, 2, 3, 16, 8


class OnGpu:
    """A tensor as the methods' checks see one on the GPU, with a CPU tensor's shape and type."""

    def __init__(self, t, device=0):
        self.t, self.is_cuda, self.device, self.index = t, True, f"cuda:{device}", device

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def arguments():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    rows = torch.zeros(T, J, dtype=torch.int32)
    return {
        "quantize": dict(X=torch.zeros(T, W)),
        "matmul_int8": dict(A=i8(T, W), scaleA=torch.ones(T), B=i8(N, W), scaleB=torch.ones(N), bias=torch.ones(N),
                            out=torch.zeros(T, N)),
        "matmul_int8_experts": dict(offsets=torch.zeros(E + 1, dtype=torch.int32), A=i8(T, W), scaleA=torch.ones(T),
                                    B=i8(E, N, W), scaleB=torch.ones(E, N), bias=torch.ones(E, N), out=torch.zeros(T, N)),
        "expert_sort": dict(ids=rows),
        "expert_dispatch": dict(X=torch.zeros(T, W), rows=rows),
        "expert_dispatch_int8": dict(X=torch.zeros(T, W), rows=rows),
        "expert_dispatch_grad": dict(dY=torch.zeros(T * J, W), rows=rows),
        "expert_combine": dict(Y=torch.zeros(T * J, W), rows=rows, weights=torch.ones(T, J)),
        "expert_combine_grad": dict(dout=torch.zeros(T, W), Y=torch.zeros(T * J, W), rows=rows, weights=torch.ones(T, J)),
    }


CASES = [(m, a) for m, args in arguments().items() for a in args]


@pytest.fixture
def g(monkeypatch):
    """The methods without a handle; reaching the library is a failure."""
    def reached(*args, **kwargs):
        raise AssertionError("the library was called")
    monkeypatch.setattr(sgemm, "_enqueue", reached)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    g = object.__new__(sgemm.Sgemm)
    g.h = None
    return g


def call(g, method, args):
    getattr(g, method)(**args, **({"experts": E} if method == "expert_sort" else {}))


@pytest.mark.parametrize("method,name", CASES)
def test_a_tensor_on_the_host_is_refused(g, method, name):
    """One of the tensors alone, and the others on the GPU."""
    args = {k: t if k == name else OnGpu(t) for k, t in arguments()[method].items()}
    with pytest.raises(ValueError, match=f"{name} must be on the GPU"):
        call(g, method, args)


@pytest.mark.parametrize("method,name", CASES)
def test_a_tensor_on_another_device_is_refused(g, method, name):
    args = {k: OnGpu(t, int(k == name)) for k, t in arguments()[method].items()}
    with pytest.raises(ValueError, match=f"{name} must be on the current device"):
        call(g, method, args)


def test_rows_of_one_column_may_have_any_column_stride():
    column = torch.zeros(1, 5).t()                     # 5 x 1, contiguous, strides (1, 5)
    assert column.is_contiguous() and column.stride(1) != 1
    sgemm._rows_of("X", column)
    assert sgemm._ld(column) == 1
    sgemm._rows_of("X", torch.zeros(5, 8)[:, 3:4])
    assert sgemm._ld(torch.zeros(5, 8)[:, 3:4]) == 8
    for bad in (torch.zeros(5, 4).t(), torch.zeros(1, 1).expand(5, 1), torch.zeros(1, 4).expand(5, 4), torch.zeros(5)):
        with pytest.raises(ValueError):
            sgemm._rows_of("X", bad)
