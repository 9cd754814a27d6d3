"""An fp8 mixture-of-experts layer from the package's operators, forward and
backward, on one GPU:

    h = dispatch(x) @ W13[e].T;  a = silu(h[:, :F]) * h[:, F:]
    y = a @ W2[e].T;             out[t] = sum over slots of weight * y

Forward and input gradients use operands quantized per block of 128
(dispatch_block, block_rows, block_tiles, grouped_mm); the weight gradients use
operands quantized per token group (colwise, grouped_wgrad).  The gate between
the two products is left to torch.

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
        step read the same copies, plain and transposed."""
        self.w13, self.w2 = gq.block_tiles(w13), gq.block_tiles(w2)

    def forward(self, x, ids, weights):
        """x bf16 (T, H); ids (T, k) expert choices (others than 0 .. E-1 are
        dropped); weights fp32 (T, k).  Returns out bf16 (T, H) and what the
        backward pass needs."""
        order = gq.sort_tokens(ids, self.experts)
        qx, sx = gq.dispatch_block(x, order.pos)
        h = gq.grouped_mm(qx, sx, *self.w13, order.offs)
        a = gated(h)
        y = gq.grouped_mm(*gq.block_rows(a), *self.w2, order.offs)
        out = gq.combine(y, order.pos, weights)
        return out, (x, weights, order, h, a, y)

    def backward(self, g, saved):
        """g bf16 (T, H).  Returns the gradients of x, weights, w13 and w2."""
        x, weights, order, h, a, y = saved
        dy, dweights = gq.combine_backward(g, y, order.pos, weights)
        da = gq.grouped_mm(*gq.block_rows(dy), *self.w2, order.offs, transpose_b=True)
        dh = gated_backward(h, da)
        dx_rows = gq.grouped_mm(*gq.block_rows(dh), *self.w13, order.offs, transpose_b=True)
        dx = gq.combine(dx_rows, order.pos)
        dw2 = weight_gradient(dy, a, order.offs)
        dw13 = weight_gradient(dh, gq.dispatch(x, order.pos), order.offs)
        return dx, dweights, dw13, dw2


def gated(h):
    left, right = h.float().chunk(2, dim=1)
    return (torch.nn.functional.silu(left) * right).to(torch.bfloat16)


def gated_backward(h, da):
    left, right = h.float().chunk(2, dim=1)
    da, s = da.float(), torch.sigmoid(left)
    dleft = da * right * s * (1 + left * (1 - s))
    return torch.cat([dleft, da * left * s], dim=1).to(torch.bfloat16)


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
