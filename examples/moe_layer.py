"""An fp8 mixture-of-experts layer from the package's operators, forward and
backward, on one GPU:

    h = dispatch(x) @ W13[e].T;  a = silu(h[:, :F]) * h[:, F:]
    y = a @ W2[e].T;             out[t] = sum over slots of weight * y

Forward and input gradients use operands quantized per block of 128
(dispatch_block, block_rows, block_tiles, grouped_gated_mm, grouped_mm); the
weight gradients use operands quantized per token group (colwise,
grouped_wgrad) and are clipped to a largest norm before a step.

    python examples/moe_layer.py        # runs it and compares with 32 bits
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_quantization_moe_gb300 as gq  # noqa: E402


class Fp8MoELayer:
    """w13 (E, 2F, H) and w2 (E, H, F) bf16 or fp32 master weights; H and F are
    multiples of 16."""

    def __init__(self, w13, w2):
        self.experts = w13.shape[0]
        self.update(w13, w2)

    def update(self, w13, w2):
        """Quantizes the weights (after an optimizer step); both products of a
        step read the same copies, plain and transposed.  The gate's and the up
        projection's rows of an expert are two matrices of it."""
        E, F2, H = w13.shape
        q, s = gq.block_tiles(w13.view(2 * E, F2 // 2, H))
        self.w13 = q.view(E, 2, F2 // 2, H), s.view(E, 2, *s.shape[1:])
        self.w2 = gq.block_tiles(w2)

    def infer(self, x, ids, weights):
        """forward without what a backward pass needs: the gated rows are
        written quantized only."""
        order = gq.sort_tokens(ids, self.experts)
        qx, sx = gq.dispatch_block(x, order.pos)
        a = gq.grouped_gated_mm(qx, sx, *self.w13, order.offs, plain=False, fp8=True)
        return gq.combine(gq.grouped_mm(a.q, a.scales, *self.w2, order.offs), order.pos, weights)

    def forward(self, x, ids, weights):
        """x bf16 (T, H); ids (T, k) expert choices (others than 0 .. E-1 are
        dropped); weights fp32 (T, k).  Returns out bf16 (T, H) and what the
        backward pass needs."""
        order = gq.sort_tokens(ids, self.experts)
        qx, sx = gq.dispatch_block(x, order.pos)
        a = gq.grouped_gated_mm(qx, sx, *self.w13, order.offs, fp8=True, keep=True)
        y = gq.grouped_mm(a.q, a.scales, *self.w2, order.offs)
        out = gq.combine(y, order.pos, weights)
        return out, (x, weights, order, a.pre, a.out, y)

    def backward(self, g, saved):
        """g bf16 (T, H).  Returns the gradients of x, weights, w13 and w2."""
        x, weights, order, pre, a, y = saved
        dy, dweights = gq.combine_backward(g, y, order.pos, weights)
        da = gq.grouped_mm(*gq.block_rows(dy), *self.w2, order.offs, transpose_b=True)
        d = gq.gated_backward(da, pre, fp8=True)
        dx_rows = gq.grouped_gated_grad(d.q, d.scales, *self.w13, order.offs)
        dx = gq.combine(dx_rows, order.pos)
        dw2 = weight_gradient(dy, a, order.offs)
        dw13 = weight_gradient(d.out.flatten(1), gq.dispatch(x, order.pos), order.offs)
        return dx, dweights, dw13, dw2

    def step(self, w13, w2, dw13, dw2, rate, max_norm):
        """A step of gradient descent on the master weights with both gradients
        clipped, in place, to a norm of max_norm together.  Returns their norm."""
        norm = gq.clip_grads([dw13, dw2], max_norm)
        w13.sub_(dw13, alpha=rate)
        w2.sub_(dw2, alpha=rate)
        self.update(w13, w2)
        return norm


def weight_gradient(grad, x, offs):
    """Per group, grad.T @ x with both operands scaled per group and column."""
    qg, sg = gq.colwise(grad, offs)
    qx, sx = gq.colwise(x, offs)
    return gq.grouped_wgrad(qg, sg.t().contiguous(), qx, sx, offs)


def plain(x, ids, weights, w13, w2, g):
    """The same layer and gradients by autograd, in the inputs' precision."""
    x, weights, w13, w2 = (t.detach().requires_grad_() for t in (x, weights, w13, w2))
    out = torch.zeros_like(x)
    for e in range(w13.shape[0]):
        token, slot = (ids == e).nonzero(as_tuple=True)
        left, right = (x[token] @ w13[e].t()).chunk(2, dim=1)
        y = (torch.nn.functional.silu(left) * right) @ w2[e].t()
        out = out.index_add(0, token, weights[token, slot, None] * y)
    return out.detach(), torch.autograd.grad(out, (x, weights, w13, w2), g)


def make_inputs(tokens, top_k, experts, hidden, width, seed=0, local=None):
    """Random inputs; with ``local`` the layer holds only the first experts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    logits = randn(tokens, experts)
    top, ids = torch.topk(logits, top_k, dim=1)
    weights = torch.softmax(top, dim=1)
    held = experts if local is None else local
    x = randn(tokens, hidden).to(torch.bfloat16)
    w13 = (randn(held, 2 * width, hidden) * hidden ** -0.5).to(torch.bfloat16)
    w2 = (randn(held, hidden, width) * width ** -0.5).to(torch.bfloat16)
    g = randn(tokens, hidden).to(torch.bfloat16)
    return x, ids, weights, w13, w2, g


def relative_errors(inputs):
    """Norm-relative differences of the layer's results from the plain ones."""
    x, ids, weights, w13, w2, g = inputs
    layer = Fp8MoELayer(w13, w2)
    out, saved = layer.forward(x, ids, weights)
    got = (out, *layer.backward(g, saved))
    gq.check_device_error()
    want_out, want = plain(x.double(), ids, weights.double(), w13.double(), w2.double(), g.double())
    names = ("out", "dx", "dweights", "dw13", "dw2")
    return {n: float((a.double() - b).norm() / b.norm())
            for n, a, b in zip(names, got, (want_out, *want))}


if __name__ == "__main__":
    gq.build()
    for name, error in relative_errors(make_inputs(2048, 4, 16, 1024, 512)).items():
        print(f"{name:9s} relative error {error:.4f}")
