"""The example's autograd functions on the CPU, over a plain stand-in for the
library's calls: first derivatives, and second ones refused -- the library's
gradients are not differentiable themselves, and autograd would take them for
constants."""
import pytest
import torch

from dense_fp32_matrix_09_gb300 import sgemm
from examples import expert_layer as ex


class Plain:
    """The calls as plain torch, without a graph, as the library's are."""
    h = None

    @staticmethod
    def expert_dispatch(x, rows):
        y = x.new_zeros(rows.numel(), x.shape[1])
        for t, j in (rows >= 0).nonzero().tolist():
            y[rows[t, j]] = x[t].detach()
        return y

    @staticmethod
    def expert_dispatch_grad(dy, rows):
        dx = dy.new_zeros(rows.shape[0], dy.shape[1])
        for t, j in (rows >= 0).nonzero().tolist():
            dx[t] += dy[rows[t, j]].detach()
        return dx

    @staticmethod
    def expert_combine(y, rows, weights):
        out = y.new_zeros(rows.shape[0], y.shape[1])
        for t, j in (rows >= 0).nonzero().tolist():
            out[t] += (weights[t, j] * y[rows[t, j]]).detach()
        return out

    @staticmethod
    def expert_combine_grad(dout, y, rows, weights):
        dy, dw = torch.zeros_like(y), torch.zeros_like(weights)
        for t, j in (rows >= 0).nonzero().tolist():
            dy[rows[t, j]] = (weights[t, j] * dout[t]).detach()
            dw[t, j] = (dout[t] * y[rows[t, j]]).sum().detach()
        return dy, dw


def run_ex(h, ta, tb, m, n, k, alpha, a, lda, sa, b, ldb, sb, beta, c, ldc, sc):
    """sgemm_run_ex on dense operands: their first m x k (k x m) and k x n (n x k) elements."""
    a, b, out = a.detach().reshape(-1), b.detach().reshape(-1), c.view(-1)
    A = a[:m * k].view(k, m).t() if ta else a[:m * k].view(m, k)
    B = b[:n * k].view(n, k).t() if tb else b[:n * k].view(k, n)
    out[:m * n] = (alpha * (A @ B)).reshape(-1)


@pytest.fixture
def pieces(monkeypatch):
    monkeypatch.setattr(sgemm, "sgemm_run_ex", run_ex)
    gen = torch.Generator().manual_seed(0)
    rows = torch.tensor([[0, 3], [-1, 1], [4, 2]], dtype=torch.int32)
    x = torch.randn(3, 4, generator=gen, requires_grad=True)
    y = torch.randn(6, 4, generator=gen, requires_grad=True)
    w = torch.rand(3, 2, generator=gen, requires_grad=True)
    W = torch.randn(2, 5, 4, generator=gen, requires_grad=True)
    bounds = [0, 2, 5]
    return {
        "dispatch": (lambda: ex.Dispatch.apply(x, rows, Plain), lambda: plain_dispatch(x, rows), [x]),
        "combine": (lambda: ex.Combine.apply(y, w, rows, Plain), lambda: plain_combine(y, w, rows), [y, w]),
        "product": (lambda: ex.ExpertProduct.apply(y, W, bounds, Plain), lambda: plain_product(y, W, bounds), [y, W]),
    }


def plain_dispatch(x, rows):
    y = x.new_zeros(rows.numel(), x.shape[1])
    for t, j in (rows >= 0).nonzero().tolist():
        y = y.index_add(0, rows[t, j].long().view(1), x[t:t + 1])
    return y


def plain_combine(y, w, rows):
    out = y.new_zeros(rows.shape[0], y.shape[1])
    for t, j in (rows >= 0).nonzero().tolist():
        out = out.index_add(0, torch.tensor([t]), w[t, j] * y[rows[t, j]][None])
    return out


def plain_product(x, W, bounds):
    done = [x[bounds[e]:bounds[e + 1]] @ W[e].t() for e in range(W.shape[0])]
    return torch.cat(done + [x.new_zeros(x.shape[0] - bounds[-1], W.shape[1])])


@pytest.mark.parametrize("name", ["dispatch", "combine", "product"])
def test_first_derivatives(pieces, name):
    mine, plain, params = pieces[name]
    dout = torch.randn(plain().shape, generator=torch.Generator().manual_seed(1))
    got, want = torch.autograd.grad(mine(), params, dout), torch.autograd.grad(plain(), params, dout)
    for a, b in zip(got, want):                        # a few products in FP32 either way
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("name", ["dispatch", "combine", "product"])
def test_second_derivatives_are_refused(pieces, name):
    mine, _, params = pieces[name]
    dout = torch.ones(mine().shape, requires_grad=True)
    first = torch.autograd.grad(mine(), params, dout, create_graph=True)
    loss = sum(t.square().sum() for t in first) + sum(t.sum() for t in params)   # (a term that is differentiable)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        loss.backward()
