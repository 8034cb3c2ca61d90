"""A mixture-of-experts layer trained with Muon on one MI355X, then decoded token
by token: the expert-layer operators as a training program calls them.

    python examples/expert_layer.py [--steps 30] [--experts 16] [--tokens 1024]

The layer learns the outputs of another layer of random weights.  Between the
forward and the backward pass it keeps its activations in 8 bits (--keep int8,
e4m3 or none); the experts' matrices are MuonPlan's, the router's weights
AdamWPlan's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_orthogonalizing_optimizer_muon_amd as M  # noqa: E402


class ExpertLayer:
    """Weights of one layer: router (experts x width, fp32), gate and up
    (experts x 2 hidden x width) and down (experts x width x hidden) in bf16."""

    def __init__(self, experts, width, hidden, k, seed, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, scale):
            return torch.randn(*shape, generator=g, device=device) * scale
        self.k = k
        self.router = draw(experts, width, scale=width ** -0.5)
        self.gate_up = draw(experts, 2 * hidden, width, scale=width ** -0.5).bfloat16()
        self.down = draw(experts, width, hidden, scale=hidden ** -0.5).bfloat16()

    def forward(self, x, keep="none"):
        """Outputs of the tokens x, and what backward() needs of this pass."""
        logits = x.float() @ self.router.t()
        r = M.route(logits, self.k)
        gu = M.grouped_matmul(x, self.gate_up, r.offsets, rows=r.rows)
        if keep == "none":
            h, kept, kept_x = M.gated(gu), gu, x
        else:
            h, kept = M.gated(gu, checkpoint=keep)
            kept_x = M.checkpoint(x, keep)
        y = M.grouped_matmul(h, self.down, r.offsets)
        return M.combine(y, r.slots, r.weights), (logits, r, kept, kept_x, y)

    def backward(self, dout, saved):
        """(router, gate_up, down) gradients and the input's by way of the experts."""
        logits, r, kept, kept_x, y = saved
        dy, dweights = M.combine_backward(dout, y, r.slots, r.weights, r.offsets)
        dgu, h = M.gated_backward(M.grouped_input_grad(dy, self.down, r.offsets), kept)
        d_down = M.grouped_weight_grad(dy, h, r.offsets)
        d_gate_up = M.grouped_weight_grad(dgu, kept_x, r.offsets, rows=r.rows)
        rows = M.grouped_input_grad(dgu, self.gate_up, r.offsets)
        dx = M.combine(rows, r.slots, torch.ones_like(r.weights))
        x = kept_x if isinstance(kept_x, torch.Tensor) else M.restore(kept_x)
        d_router = M.route_backward(dweights, logits, r).t() @ x.float()
        return (d_router, d_gate_up, d_down), dx


def train(steps=30, experts=16, tokens=1024, width=256, hidden=192, k=2, keep="int8", lr=0.02, report=None):
    """Losses of the steps, and the layer."""
    teacher, layer = (ExpertLayer(experts, width, hidden, k, seed) for seed in (1, 2))
    matrices = [*layer.gate_up, *layer.down]      # each expert's, in place
    shapes = [tuple(m.shape) for m in matrices]
    g = torch.Generator(device="cuda").manual_seed(3)
    momenta = [torch.zeros(s, device="cuda") for s in shapes]
    moments = [torch.zeros_like(layer.router) for _ in range(2)]
    losses = []
    with M.MuonPlan(shapes, "bf16", tune="off") as muon:
        adamw = M.AdamWPlan([layer.router.numel()], "f32")
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        want = teacher.forward(x)[0].float()
        for step in range(1, steps + 1):
            out, saved = layer.forward(x, keep)
            off = out.float() - want
            losses.append(float(off.square().mean()))
            grads, _ = layer.backward((off * (2 / off.numel())).bfloat16(), saved)
            muon.step(matrices, [*grads[1], *grads[2]], momenta, lr=lr, wd=0.0)
            adamw.step([layer.router], [grads[0].contiguous()], [moments[0]], [moments[1]], lr=1e-3, step=step)
            if report and (step == 1 or step % 10 == 0):
                report(f"step {step}: loss {losses[-1]:.5f}")
        adamw.close()
    return losses, layer, x


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--keep", choices=["none", "int8", "e4m3"], default="int8")
    a = p.parse_args()
    losses, layer, x = train(a.steps, a.experts, a.tokens, keep=a.keep, report=lambda s: print(s, flush=True))
    whole = layer.forward(x)[0]
    single = torch.cat([layer.forward(x[i:i + 1])[0] for i in range(8)])
    off = (single.float() - whole[:8].float()).abs().max() / whole[:8].float().abs().max()
    print(f"eight tokens decoded one by one: off by {float(off):.1e} of the largest output")


if __name__ == "__main__":
    main()
