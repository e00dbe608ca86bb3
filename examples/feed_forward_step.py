"""Training steps of one dense feed-forward layer, from the residual stream to the Muon step.

    python examples/feed_forward_step.py [--steps 8] [--tokens 2048] [--check] [--fp8]

The layer: x + down(silu(n gate) * (n up)), with n the layer norm of x.  All parameters live in one
flat fp32 buffer (the norm's weight and bias, then gate, up and down), with a bf16 copy for the
products.  A step uses the library from end to end:

    muon_layer_norm(_grad)  the norm, with the statistics its gradient takes
    muon_gated_mm           both projections and the activation in one kernel
    muon_grouped_mm         the down projection
    muon_gated_mm_grad      back through the down projection and the activation
    muon_grouped_mm_sum     back through both projections, summed before the rounding
    muon_grouped_wgrad      weight gradients, straight into the flat gradient buffer
    muon_grad_norm          the norm over all gradients, and the clipping coefficient
    muon_step_scaled        Muon on the matrices, clipped by that coefficient

--fp8 also runs the trained layer forward with 8-bit products (muon_quantize_weights once,
muon_quantize_rows and muon_grouped_mm_fp8 for each product) and compares the outputs.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from muon_optimizer_step_gb300 import capi  # noqa: E402


class FeedForward:
    """One layer's parameters, gradients and optimizer state in flat buffers."""

    def __init__(self, hidden, inner, seed=0):
        self.hidden, self.inner = hidden, inner
        shapes = [(hidden, 1), (hidden, 1), (hidden, inner), (hidden, inner), (inner, hidden)]
        self.layout = capi.muon_layout_create(shapes, 1, capi.MUON_NS_BF16, [False, False, True, True, True])
        self.workspace = capi.workspace_tensor(self.layout)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        n = self.layout.numel
        self.weights = torch.randn(n, generator=gen, device="cuda") * hidden ** -0.5
        self.weights[:hidden] = 1.0
        self.weights[hidden:2 * hidden] = 0.0
        self.grads = torch.zeros(n, device="cuda")
        self.momentum = torch.zeros(n, device="cuda")
        self.half = torch.empty(n, device="cuda", dtype=torch.bfloat16)
        self.norm = torch.empty(2, device="cuda")

    def views(self, flat):
        """norm weight and bias (hidden), gate, up (1, hidden, inner) and down (1, inner, hidden)."""
        h, f = self.hidden, self.inner
        at = 2 * h
        return (flat[:h], flat[h:at], flat[at:at + h * f].view(1, h, f),
                flat[at + h * f:at + 2 * h * f].view(1, h, f), flat[at + 2 * h * f:].view(1, f, h))

    def loss_and_grads(self, x, target):
        """The mean squared error of the layer on x (tokens, hidden; bfloat16); fills self.grads and
        returns the loss and the gradient with respect to x."""
        tokens = x.shape[0]
        self.half.copy_(self.weights)
        weight, bias = self.views(self.weights)[:2]
        _, _, gate, up, down = self.views(self.half)
        offsets = torch.tensor([0, tokens], dtype=torch.int64, device=x.device)

        def new(width):
            return torch.empty(tokens, width, device=x.device, dtype=torch.bfloat16)

        mean, rstd = torch.empty(2, tokens, device=x.device)
        n, act, g, u, y = new(self.hidden), new(self.inner), new(self.inner), new(self.inner), new(self.hidden)
        capi.muon_layer_norm(x, weight, bias, n, mean=mean, rstd=rstd)
        capi.muon_gated_mm(n, gate, up, None, act, gate=g, up=u)
        capi.muon_grouped_mm(act, down, offsets, y)
        error = x.float() + y.float() - target

        dout = error * (2.0 / error.numel())
        dy = dout.bfloat16()
        dg, du, dn, dx = new(self.inner), new(self.inner), new(self.hidden), new(self.hidden)
        dweight, dbias, dgate, dup, ddown = self.views(self.grads)
        # (act is computed again here: a training run need not keep it from the forward pass.)
        capi.muon_gated_mm_grad(dy, down, None, g, u, dg, du, out=act, trans_w=True)
        capi.muon_grouped_wgrad(act, dy, offsets, ddown)
        capi.muon_grouped_wgrad(n, dg, offsets, dgate)
        capi.muon_grouped_wgrad(n, du, offsets, dup)
        capi.muon_grouped_mm_sum(dg, gate, du, up, None, dn, trans_w=True)
        capi.muon_layer_norm_grad(dn, x, weight, mean, rstd, dx, dweight, dbias)
        return error.square().mean(), dout + dx.float()

    def forward_fp8(self, x):
        """The layer's output with 8-bit products; the weights would be kept between calls."""
        tokens, e4m3 = x.shape[0], torch.float8_e4m3fn
        self.half.copy_(self.weights)
        weight, bias = self.views(self.weights)[:2]

        def quantized_weight(w):
            _, k, n = w.shape
            q = torch.empty(1, n, k + -k % 16, dtype=torch.uint8, device=x.device).view(e4m3)[..., :k]
            scale = torch.empty(1, -(-n // capi.FP8_BLOCK), -(-k // capi.FP8_BLOCK), device=x.device)
            capi.muon_quantize_weights(w, q, scale, transpose=True)
            return q, scale

        def product(a, weight8):
            k = a.shape[1]
            q = torch.empty(tokens, k + -k % 16, dtype=torch.uint8, device=x.device).view(e4m3)[:, :k]
            scale = torch.empty(-(-k // capi.FP8_BLOCK), tokens, device=x.device)
            y = torch.empty(tokens, weight8[0].shape[1], dtype=torch.bfloat16, device=x.device)
            capi.muon_quantize_rows(a, q, scale)
            capi.muon_grouped_mm_fp8(q, scale, *weight8, None, y)
            return y

        gate, up, down = (quantized_weight(w) for w in self.views(self.half)[2:])
        n = torch.empty_like(x)
        capi.muon_layer_norm(x, weight, bias, n)
        g, u = product(n, gate), product(n, up)
        act = torch.empty_like(g)
        capi.muon_swiglu(g, u, act)
        return x.float() + product(act, down).float()

    def step(self, lr, max_norm):
        """Clips by the global norm and steps: Muon on the matrices, plain descent on the norm."""
        capi.muon_grad_norm(capi.layout_grads(self.layout, self.grads), max_norm, self.norm)
        capi.muon_step_scaled([self.weights], [self.grads], [self.momentum], self.layout,
                              self.workspace, [(lr, 0.0, 0.95, True)], self.norm[1:])
        for w, g in zip(self.views(self.weights)[:2], self.views(self.grads)[:2]):
            w.sub_(g * (lr * self.norm[1]))


def reference_grads(layer, x, target):
    """The same loss and gradients by torch's automatic differentiation, in 64 bits, with the layer's
    bf16 matrices; and the layer's output."""
    leaves = [t.double().requires_grad_(True) for t in
              (*layer.views(layer.weights)[:2], *layer.views(layer.weights.bfloat16())[2:], x)]
    weight, bias, gate, up, down, xd = leaves
    n = torch.nn.functional.layer_norm(xd, (layer.hidden,), weight, bias, 1e-5)
    out = xd + (torch.nn.functional.silu(n @ gate[0]) * (n @ up[0])) @ down[0]
    loss = (out - target.double()).square().mean()
    return loss, torch.autograd.grad(loss, leaves), out.detach()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=1408)
    ap.add_argument("--lr", type=float, default=0.02)
    ap.add_argument("--max-norm", type=float, default=0.02)
    ap.add_argument("--check", action="store_true", help="compare the gradients with 64 bits first")
    ap.add_argument("--fp8", action="store_true", help="compare the 8-bit forward pass with 64 bits at the end")
    a = ap.parse_args(argv)
    layer = FeedForward(a.hidden, a.inner)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda")
    worst = off = None
    if a.check:
        loss, dx = layer.loss_and_grads(x, target)
        want, grads, _ = reference_grads(layer, x, target)
        got = [*layer.views(layer.grads), dx]
        worst = max(float((t.double() - w).norm() / w.norm()) for t, w in zip(got, grads))
        print(f"loss {float(loss):.6f} (64 bits {float(want.detach()):.6f}), "
              f"gradients within {worst:.2e} of 64 bits")
    losses = []
    for i in range(a.steps):
        loss, _ = layer.loss_and_grads(x, target)
        layer.step(a.lr, a.max_norm)
        losses.append((loss, layer.norm.clone()))
    if a.fp8:
        out = reference_grads(layer, x, target)[2]
        off = float(((layer.forward_fp8(x).double() - out).norm() / (out - x.double()).norm()))
        print(f"8-bit forward pass within {off:.2e} of 64 bits (of what the layer adds to its input)")
    capi.muon_check()
    for i, (loss, norm) in enumerate(losses):
        print(f"step {i}: loss {float(loss):.6f}, gradient norm {float(norm[0]):.4f}, "
              f"clipped by {float(norm[1]):.4f}")
    return worst, off


if __name__ == "__main__":
    main()
