"""Trains one expert layer on a random target: router, routing, grouped
projections, and AdamW with 8-bit moments.

    y = combine(silu(dispatch(x) W1[e]^T) W2[e]^T),  loss = mean (y - target)^2

The expert weights are FP32 masters with BF16 copies that the products read;
their gradients come from the grouped weight gradient in FP32.

    python examples/expert_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_bf16_projection_amd as dpg  # noqa: E402


class ExpertLayer:
    """Weights, 8-bit optimizer state and one training step."""

    def __init__(self, experts, hidden, inner, top_k, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        shapes = [(experts, hidden), (experts, inner, hidden), (experts, hidden, inner)]  # router, W1, W2
        self.masters = [(torch.randn(s, generator=g) * s[-1] ** -0.5).to(device) for s in shapes]
        self.weights = [m.to(torch.bfloat16) for m in self.masters]
        self.moments = [[torch.zeros(s, device=device).to(torch.float8_e4m3fn) for s in shapes] for _ in range(2)]
        blocks = [-(-m.numel() // dpg.ADAMW_BLOCK) for m in self.masters]
        self.scales = [[torch.ones(b, device=device) for b in blocks] for _ in range(2)]
        self.top_k, self.step_count = top_k, 0

    def forward(self, x):
        """Output of the layer and what the gradients need."""
        logits = dpg.dpg_router_forward(x.float(), self.masters[0])
        r = dpg.dpg_route(logits, self.top_k)
        xs = dpg.dpg_dispatch(x, r.positions, r.offsets)
        a = dpg.dpg_grouped_forward(xs, self.weights[1], r.offsets)
        h = torch.nn.functional.silu(a)
        ys = dpg.dpg_grouped_forward(h, self.weights[2], r.offsets)
        return dpg.dpg_combine(ys, r.positions, r.offsets, r.weights), (logits, r, xs, a, h, ys)

    def gradients(self, x, dy, saved):
        """FP32 gradients of the router, W1 and W2, and the BF16 gradient of x
        (through the experts; the router's part is added by the caller's layer)."""
        logits, r, xs, a, h, ys = saved
        dys, dweights = dpg.dpg_combine_dgrad(dy, ys, r.positions, r.offsets, r.weights)
        dw2 = dpg.dpg_grouped_wgrad(dys, h, r.offsets, out_dtype=torch.float32)
        dh = dpg.dpg_grouped_dgrad(dys, self.weights[2], r.offsets)
        s = torch.sigmoid(a.float())
        da = (dh.float() * s * (1 + a.float() * (1 - s))).to(torch.bfloat16)
        dw1 = dpg.dpg_grouped_wgrad(da, xs, r.offsets, out_dtype=torch.float32)
        dx = dpg.dpg_combine(dpg.dpg_grouped_dgrad(da, self.weights[1], r.offsets), r.positions, r.offsets)
        dlogits = dpg.dpg_route_dgrad(logits, r.experts, r.weights, dweights)
        return [dpg.dpg_router_wgrad(dlogits, x.float()), dw1, dw2], dx

    def train_step(self, x, target, lr=2e-3):
        y, saved = self.forward(x)
        error = y.float() - target
        loss = error.square().mean()
        grads, _ = self.gradients(x, (error * (2 / error.numel())).to(torch.bfloat16), saved)
        self.step_count += 1
        norm = torch.stack([g.norm() for g in grads]).norm()
        dpg.dpg_adamw(self.masters, grads, *self.moments, lr=lr, beta2=0.95, weight_decay=0.0, step=self.step_count,
                      copies=self.weights, avg_scales=self.scales[0], sq_scales=self.scales[1],
                      grad_scale=(1.0 / norm).clamp(max=1.0).reshape(1), seed=self.step_count)
        return loss


def main(steps=50, tokens=512, experts=16, hidden=256, inner=512, top_k=4):
    layer = ExpertLayer(experts, hidden, inner, top_k)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16).cuda()
    target = torch.randn(tokens, hidden, generator=g).cuda()
    losses = [float(layer.train_step(x, target)) for _ in range(steps)]
    for i in range(0, steps, max(1, steps // 10)):
        print("step %3d  loss %.4f" % (i + 1, losses[i]))
    print("step %3d  loss %.4f" % (steps, losses[-1]))
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 50)
