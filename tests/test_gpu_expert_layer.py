"""The mixture-of-experts example end to end, and the tensor methods' checks.

Tolerances.  Served: weights and activations carry 7 bits and a sign; each of the
four quantized operands errs by at most half a step, 1/254 of its row's largest
value, which for normal rows of 64 and more is at most 1/254 * 4.5 standard
deviations = 1.8 % of a row's root mean square, and uniformly distributed 1.8 % /
sqrt(3) = 1.0 % in the mean: 2.1 % for the four together, in the output's norm
(the product of two independent rows averages the errors as it does the values,
and silu's slope is at most 1.1); the limit is twice that, 5 %, BF16 included.  Trained: FP32 products
of at most 128 terms and their gradients, 1e-5 of the norm (128 * 2^-24 = 8e-6)."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from examples import expert_layer as ex

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_fp32_matrix_09_gb300 import build
    build.build()
    with sgemm.Sgemm() as handle:
        yield handle
        assert handle.device_status() == sgemm.OK


def layer(tokens, width, hidden, experts, choices, dropped, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, width, generator=gen, device="cuda")
    up = torch.randn(experts, hidden, width, generator=gen, device="cuda") / width ** 0.5
    down = torch.randn(experts, width, hidden, generator=gen, device="cuda") / hidden ** 0.5
    ids, weights = ex.route(torch.randn(tokens, experts, generator=gen, device="cuda"), choices)
    if dropped:
        ids[::3, 0] = -1
        ids[-1] = -1            # a token whose choices are all dropped
    return x, ids, weights, up, down


@pytest.mark.parametrize("tokens,choices,dropped", [(1, 2, False), (7, 2, True), (200, 2, False), (300, 4, True)])
def test_served(g, tokens, choices, dropped):
    x, ids, weights, up, down = layer(tokens, 128, 96, 6, choices, dropped)
    want = ex.plain_forward(x.double(), ids, weights.double(), up.double(), down.double())
    got = ex.ServedExperts(g, up, down)(x.bfloat16(), ids, weights)
    assert float((got.double() - want).norm()) <= 0.05 * float(want.norm())
    if dropped:
        assert bool((got[-1] == 0).all())


@pytest.mark.parametrize("tokens,choices,dropped", [(5, 2, False), (64, 3, True)])
def test_trained_gradients(g, tokens, choices, dropped):
    x, ids, weights, up, down = layer(tokens, 64, 128, 5, choices, dropped, seed=1)
    params = [t.clone().requires_grad_() for t in (x, weights, up, down)]
    out = ex.trained_forward(g, params[0], ids, *params[1:])
    exact = [t.double().requires_grad_() for t in (x, weights, up, down)]
    want = ex.plain_forward(exact[0], ids, *exact[1:])
    dout = torch.randn(out.shape, device="cuda")
    out.backward(dout)
    want.backward(dout.double())
    out, want = out.detach(), want.detach()
    assert float((out.double() - want).norm()) <= 1e-5 * float(want.norm())
    for p, q in zip(params, exact):
        assert float((p.grad.double() - q.grad).norm()) <= 1e-5 * float(q.grad.norm())


def test_example_runs(g, capsys):
    ex.main()
    assert "one step of gradient descent" in capsys.readouterr().out


def test_tensor_methods_check_their_arguments(g):
    a = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    b = torch.zeros(8, 32, dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    assert g.matmul_int8(a, sa, b, sb).dtype == torch.bfloat16
    assert g.matmul_int8(a[:, ::1][1:3], sa[1:3], b, sb, out_dtype=torch.float32).shape == (2, 8)
    rows = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: g.matmul_int8(a.float(), sa, b, sb), lambda: g.matmul_int8(a, sa, b[:, :16].contiguous(), sb),
                lambda: g.matmul_int8(a, sb, b, sb), lambda: g.matmul_int8(a, sa.double(), b, sb),
                lambda: g.matmul_int8(a, sa, b, sb, bias=sa), lambda: g.matmul_int8(a, sa, b, sb, out_dtype=torch.int32),
                lambda: g.matmul_int8(a, sa, b, sb, out=torch.zeros(4, 9, device="cuda")),
                lambda: g.matmul_int8(a.t(), sa, b, sb), lambda: g.quantize(a), lambda: g.quantize(x.t()),
                lambda: g.quantize(x[:1].expand(3, 16)),
                lambda: g.expert_sort(rows.long(), 4), lambda: g.expert_dispatch(x, rows[:3]),
                lambda: g.expert_combine(x, rows, torch.ones(4, 2, device="cuda")),
                lambda: g.expert_combine(torch.zeros(8, 16, device="cuda"), rows, torch.ones(2, 4, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
