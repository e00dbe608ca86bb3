"""Training steps of one mixture-of-experts layer, from the tokens to the Muon step.

    python examples/expert_layer_step.py [--steps 8] [--tokens 2048] [--check]

The layer: a softmax router sends every token to its `top` best experts; each expert is
down(silu(x gate) * (x up)), weighted by the router.  All parameters live in one flat fp32
buffer (router, then gate, up and down of every expert), with a bf16 copy for the products.
A step uses the library from end to end:

    muon_grouped_mm     x gate, x up, act down, and backward the same with trans_w
    muon_swiglu(_grad)  the activation with the router's weight of each row, and its gradient
    muon_grouped_wgrad  weight gradients, straight into the flat gradient buffer
    muon_grad_norm      the norm over all gradients, and the clipping coefficient
    muon_step_scaled    Muon on the experts' matrices, clipped by that coefficient

Routing, gathering and the router's own (small) gradient are plain torch.  The row offsets
stay on the GPU: no step waits for the host.
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


class ExpertLayer:
    """One layer's parameters, gradients and optimizer state in flat buffers."""

    def __init__(self, hidden, inner, experts, top, seed=0):
        self.hidden, self.inner, self.experts, self.top = hidden, inner, experts, top
        shapes = [(hidden, experts)] + [(hidden, inner), (hidden, inner), (inner, hidden)] * experts
        self.layout = capi.muon_layout_create(shapes, 1, capi.MUON_NS_BF16,
                                              [False] + [True] * (3 * experts))
        self.workspace = capi.workspace_tensor(self.layout)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        n = self.layout.numel
        self.weights = torch.randn(n, generator=gen, device="cuda") * hidden ** -0.5
        self.grads = torch.zeros(n, device="cuda")
        self.momentum = torch.zeros(n, device="cuda")
        self.half = torch.empty(n, device="cuda", dtype=torch.bfloat16)
        self.norm = torch.empty(2, device="cuda")

    def views(self, flat):
        """router (hidden, experts) and gate, up, down (experts, rows, cols) of a flat buffer."""
        h, f, e = self.hidden, self.inner, self.experts
        at, step = h * e, 3 * h * f
        return (flat[:at].view(h, e),
                flat.as_strided((e, h, f), (step, f, 1), at),
                flat.as_strided((e, h, f), (step, f, 1), at + h * f),
                flat.as_strided((e, f, h), (step, h, 1), at + 2 * h * f))

    def loss_and_grads(self, x, target):
        """The mean squared error of the layer on x (tokens, hidden); fills self.grads and
        returns the loss and the gradient with respect to x."""
        tokens = x.shape[0]
        self.half.copy_(self.weights)
        _, gate, up, down = self.views(self.half)
        router = self.views(self.weights)[0].detach().requires_grad_(True)
        xr = x.float().requires_grad_(True)
        prob, pick = (xr @ router).softmax(1).topk(self.top, dim=1)

        # rows sorted by expert
        order = pick.reshape(-1).argsort(stable=True)
        token = order // self.top
        counts = torch.zeros(self.experts, dtype=torch.int64, device=x.device)
        counts.scatter_add_(0, pick.reshape(-1), torch.ones_like(order))
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        weight = prob.reshape(-1)[order]
        p = weight.detach().contiguous()
        rows = x[token]

        def new(width):
            return torch.empty(tokens * self.top, width, device=x.device, dtype=torch.bfloat16)

        g, u, act, y = new(self.inner), new(self.inner), new(self.inner), new(self.hidden)
        capi.muon_grouped_mm(rows, gate, offsets, g)
        capi.muon_grouped_mm(rows, up, offsets, u)
        capi.muon_swiglu(g, u, act, row_weight=p)
        capi.muon_grouped_mm(act, down, offsets, y)
        out = torch.zeros(tokens, self.hidden, device=x.device).index_add_(0, token, y.float())

        error = out - target
        dy = (error * (2.0 / error.numel()))[token].bfloat16()
        dact, dg, du = new(self.inner), new(self.inner), new(self.inner)
        dp = torch.empty_like(p)
        _, dgate, dup, ddown = self.views(self.grads)
        capi.muon_grouped_mm(dy, down, offsets, dact, trans_w=True)
        capi.muon_grouped_wgrad(act, dy, offsets, ddown)
        capi.muon_swiglu_grad(dact, g, u, dg, du, row_weight=p, d_row_weight=dp)
        capi.muon_grouped_wgrad(rows, dg, offsets, dgate)
        capi.muon_grouped_wgrad(rows, du, offsets, dup)
        dx_gate, dx_up = new(self.hidden), new(self.hidden)
        capi.muon_grouped_mm(dg, gate, offsets, dx_gate, trans_w=True)
        capi.muon_grouped_mm(du, up, offsets, dx_up, trans_w=True)
        drouter, dx = torch.autograd.grad(weight, (router, xr), dp)
        self.views(self.grads)[0].copy_(drouter)
        dx = dx.index_add(0, token, dx_gate.float() + dx_up.float())
        return error.square().mean(), dx

    def step(self, lr, max_norm):
        """Clips by the global norm and steps: Muon on the experts, plain descent on the router."""
        capi.muon_grad_norm(capi.layout_grads(self.layout, self.grads), max_norm, self.norm)
        capi.muon_step_scaled([self.weights], [self.grads], [self.momentum], self.layout,
                              self.workspace, [(lr, 0.0, 0.95, True)], self.norm[1:])
        router, grad = self.views(self.weights)[0], self.views(self.grads)[0]
        router.sub_(grad * (lr * self.norm[1]))


def reference_grads(layer, x, target):
    """The same loss and gradients by torch's automatic differentiation, in 64 bits, with the
    layer's bf16 experts and its choice of experts."""
    router = layer.views(layer.weights)[0].double().requires_grad_(True)
    gate, up, down = [t.double().requires_grad_(True) for t in layer.views(layer.weights.bfloat16())[1:]]
    xd = x.double().requires_grad_(True)
    pick = (x.float() @ layer.views(layer.weights)[0]).softmax(1).topk(layer.top, dim=1).indices
    prob = (xd @ router).softmax(1).gather(1, pick)
    out = 0
    for j in range(layer.top):
        hidden = torch.einsum("th,ehf->tef", xd, gate), torch.einsum("th,ehf->tef", xd, up)
        one = torch.nn.functional.one_hot(pick[:, j], layer.experts).double()
        act = (torch.nn.functional.silu(hidden[0]) * hidden[1]) * one[:, :, None]
        out = out + prob[:, j:j + 1] * torch.einsum("tef,efh->th", act, down)
    loss = (out - target.double()).square().mean()
    return loss, torch.autograd.grad(loss, (router, gate, up, down, xd))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=704)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=4)
    ap.add_argument("--lr", type=float, default=0.02)
    ap.add_argument("--max-norm", type=float, default=0.02)
    ap.add_argument("--check", action="store_true", help="compare the gradients with 64 bits first")
    a = ap.parse_args(argv)
    layer = ExpertLayer(a.hidden, a.inner, a.experts, a.top)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda")
    worst = None
    if a.check:
        loss, dx = layer.loss_and_grads(x, target)
        want, grads = reference_grads(layer, x, target)
        got = [*layer.views(layer.grads), dx]
        worst = max(float((t.double() - w).norm() / w.norm()) for t, w in zip(got, grads))
        print(f"loss {float(loss):.6f} (64 bits {float(want.detach()):.6f}), "
              f"gradients within {worst:.2e} of 64 bits")
    losses = []
    for i in range(a.steps):
        loss, _ = layer.loss_and_grads(x, target)
        layer.step(a.lr, a.max_norm)
        losses.append((loss, layer.norm.clone()))
    capi.muon_check()
    for i, (loss, norm) in enumerate(losses):
        print(f"step {i}: loss {float(loss):.6f}, gradient norm {float(norm[0]):.4f}, "
              f"clipped by {float(norm[1]):.4f}")
    return [float(loss) for loss, _ in losses], worst


if __name__ == "__main__":
    main()
