"""A mixture-of-experts layer on the library's calls.

Serving: the router's choices are sorted by expert, the tokens' rows are moved to
their experts and quantized on the way, two int8 products with each expert's
weights (an activation between them, quantized again) and the weighted way back.

Training: dispatch and combine as autograd functions around FP32 products of
each expert's rows (sgemm_run_ex), one step of gradient descent on a small target.

The gradients are the library's results, not differentiable themselves: a second
derivative is refused.

    python -m examples.expert_layer            # needs a GB300 and the built library
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from dense_fp32_matrix_09_gb300 import sgemm


def route(logits, choices):
    """(ids, weights): each token's experts and the softmax over their logits."""
    top = logits.topk(choices, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values.float(), dim=1).contiguous()


class ServedExperts:
    """Weights quantized once, one scale a channel; __call__ is one forward pass."""

    def __init__(self, g: sgemm.Sgemm, up, down):
        self.g = g
        experts, hidden, width = up.shape                       # up: E x hidden x width, down: E x width x hidden
        self.up, self.up_scale = (t.reshape(experts, hidden, -1) for t in g.quantize(up.reshape(-1, width)))
        self.down, self.down_scale = (t.reshape(experts, width, -1) for t in g.quantize(down.reshape(-1, hidden)))
        self.up_scale, self.down_scale = self.up_scale.squeeze(2).contiguous(), self.down_scale.squeeze(2).contiguous()
        self.up, self.down = self.up.contiguous(), self.down.contiguous()

    def __call__(self, x, ids, weights):
        g = self.g
        offsets, rows, _ = g.expert_sort(ids, self.up.shape[0])
        q, scale = g.expert_dispatch_int8(x, rows)
        h = g.matmul_int8_experts(offsets, q, scale, self.up, self.up_scale, out_dtype=x.dtype)
        q, scale = g.quantize(torch.nn.functional.silu(h))
        y = g.matmul_int8_experts(offsets, q, scale, self.down, self.down_scale, out_dtype=x.dtype)
        return g.expert_combine(y, rows, weights)


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, g):
        ctx.g, ctx.rows = g, rows
        return g.expert_dispatch(x, rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return ctx.g.expert_dispatch_grad(dy.contiguous(), ctx.rows), None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, rows, g):
        ctx.g, ctx.rows = g, rows
        ctx.save_for_backward(y, weights)
        return g.expert_combine(y, rows, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, weights = ctx.saved_tensors
        dy, dweights = ctx.g.expert_combine_grad(dout.contiguous(), y, ctx.rows, weights)
        return dy, dweights, None, None


class ExpertProduct(torch.autograd.Function):
    """y[rows of e] = x[rows of e] @ w[e].T in FP32, one sgemm_run_ex an expert and direction."""

    @staticmethod
    def forward(ctx, x, w, bounds, g):
        ctx.g, ctx.bounds = g, bounds
        ctx.save_for_backward(x, w)
        (experts, n, k), y = w.shape, x.new_zeros(x.shape[0], w.shape[1])
        for e in range(experts):
            r, m = bounds[e], bounds[e + 1] - bounds[e]
            sgemm.sgemm_run_ex(g.h, 0, 1, m, n, k, 1.0, x[r:], k, 0, w[e], k, 0, 0.0, y[r:], n, 0)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (x, w), g, bounds = ctx.saved_tensors, ctx.g, ctx.bounds
        dy = dy.contiguous()
        (experts, n, k), dx, dw = w.shape, torch.zeros_like(x), torch.zeros_like(w)
        for e in range(experts):
            r, m = bounds[e], bounds[e + 1] - bounds[e]
            sgemm.sgemm_run_ex(g.h, 0, 0, m, k, n, 1.0, dy[r:], n, 0, w[e], k, 0, 0.0, dx[r:], k, 0)
            sgemm.sgemm_run_ex(g.h, 1, 0, n, k, m, 1.0, dy[r:], n, 0, x[r:], k, 0, 0.0, dw[e], k, 0)
        return dx, dw, None, None


def trained_forward(g, x, ids, weights, up, down):
    """The same layer in FP32, differentiable in x, weights, up and down."""
    offsets, rows, _ = g.expert_sort(ids, up.shape[0])
    bounds = offsets.tolist()
    h = ExpertProduct.apply(Dispatch.apply(x, rows, g), up, bounds, g)
    y = ExpertProduct.apply(torch.nn.functional.silu(h), down, bounds, g)
    return Combine.apply(y, weights, rows, g)


def plain_forward(x, ids, weights, up, down):
    """In whatever precision the inputs have, with torch alone."""
    out = torch.zeros_like(x)
    for e in range(up.shape[0]):
        token, j = (ids == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[token] @ up[e].T) @ down[e].T
        out = out.index_add(0, token, y * weights[token, j].to(x.dtype)[:, None])
    return out


def main() -> None:
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    tokens, width, hidden, experts, choices = 200, 256, 512, 8, 2
    x, logits = randn(tokens, width), randn(tokens, experts)
    up, down = randn(experts, hidden, width) / width ** 0.5, randn(experts, width, hidden) / hidden ** 0.5
    ids, weights = route(logits, choices)
    with sgemm.Sgemm() as g:
        want = plain_forward(x.double(), ids, weights.double(), up.double(), down.double())
        served = ServedExperts(g, up, down)(x.bfloat16(), ids, weights)
        print(f"served (int8): relative error {float((served.double() - want).norm() / want.norm()):.4f}")
        params = [t.clone().requires_grad_() for t in (x, weights, up, down)]
        out = trained_forward(g, params[0], ids, *params[1:])
        print(f"trained (FP32): relative error {float((out.detach().double() - want).norm() / want.norm()):.2e}")
        loss = out.square().mean()
        loss.backward()
        with torch.no_grad():
            stepped = [t - 0.5 * t.grad for t in params]
            after = trained_forward(g, stepped[0], ids, *stepped[1:]).square().mean()
        print(f"one step of gradient descent: loss {float(loss.detach()):.6f} -> {float(after):.6f}")
        if g.device_status() != sgemm.OK:
            raise RuntimeError(sgemm.status_string(g.device_status()))


if __name__ == "__main__":
    main()
