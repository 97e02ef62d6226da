"""Trains a residual block that mixes tokens with a gated recurrence: the running
mean of a sequence, from its noisy values.

    n, stream = add_layer_norm(dropout(y), stream)      y: the output of the block before
    h = recurrence(n W_gate^T, n W_in^T)                along each sequence
    y = h W_out^T

Weights are FP32 masters with BF16 copies that the products read, and AdamW's
moments are 8-bit.  The dropout's step is counted on the device.

    python examples/recurrent_block.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_bf16_projection_amd as dpg  # noqa: E402
from deterministic_bf16_projection_amd import autograd as dag  # noqa: E402


class RecurrentBlocks:
    """`layers` blocks over an FP32 residual stream, their optimizer state and one
    training step.  names: the masters' order."""

    names = ("w_norm", "b_norm", "w_gate", "w_in", "w_out")

    def __init__(self, layers, hidden, inner, p=0.1, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.layers, self.p, self.seed = layers, p, seed
        self.masters, self.copies = [], []
        for _ in range(layers):
            shapes = [(hidden,), (hidden,), (inner, hidden), (inner, hidden), (hidden, inner)]
            values = [torch.ones(hidden), torch.zeros(hidden)]
            values += [torch.randn(s, generator=g) * s[-1] ** -0.5 for s in shapes[2:]]
            self.masters += [v.to(device) for v in values]
        self.masters += [torch.ones(hidden, device=device), torch.zeros(hidden, device=device)]
        self.copies = [m.to(torch.bfloat16) for m in self.masters]
        self.moments = [[torch.zeros_like(m).to(torch.float8_e4m3fn) for m in self.masters] for _ in range(2)]
        self.scales = [[torch.ones(-(-m.numel() // dpg.ADAMW_BLOCK), device=device) for m in self.masters]
                       for _ in range(2)]
        self.step = torch.zeros(1, dtype=torch.int64, device=device)
        self.count = 0

    def forward(self, x, leaves, training=True):
        """leaves: norms in FP32, projections in BF16, in the masters' order."""
        p = self.p if training else 0.0
        stream, y = x.float(), torch.zeros_like(x)
        for i in range(self.layers):
            w_norm, b_norm, w_gate, w_in, w_out = leaves[5 * i:5 * i + 5]
            n, stream = dag.add_layer_norm(y, stream, w_norm, b_norm, p=p, seed=self.seed + i, step=self.step,
                                           out_dtype=torch.bfloat16)
            h, _ = dag.recurrence(dag.projection(n, w_gate), dag.projection(n, w_in))
            y = dag.projection(h, w_out)
        out, _ = dag.add_layer_norm(y, stream, leaves[-2], leaves[-1], p=p, seed=self.seed + self.layers,
                                    step=self.step, out_dtype=torch.float32)
        return out

    def leaves(self):
        return [(m if m.dim() == 1 else c).detach().requires_grad_(True) for m, c in zip(self.masters, self.copies)]

    def train_step(self, x, target, lr=3e-3):
        leaves = self.leaves()
        loss = (self.forward(x, leaves) - target).square().mean()
        grads = [g.float() for g in torch.autograd.grad(loss, leaves)]
        self.count += 1
        norm = torch.stack([g.norm() for g in grads]).norm()
        dpg.dpg_adamw(self.masters, grads, *self.moments, lr=lr, beta2=0.95, weight_decay=0.0, step=self.count,
                      copies=self.copies, avg_scales=self.scales[0], sq_scales=self.scales[1],
                      grad_scale=(1.0 / norm).clamp(max=1.0).reshape(1), seed=self.count)
        self.step += 1
        return loss.detach()


def main(steps=50, batch=8, length=256, layers=2, hidden=128, inner=256):
    model = RecurrentBlocks(layers, hidden, inner)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(batch, length, hidden, generator=g)
    target = x.cumsum(1) / torch.arange(1, length + 1)[None, :, None] * 4
    x, target = x.to(torch.bfloat16).cuda(), target.cuda()
    losses = [float(model.train_step(x, target)) for _ in range(steps)]
    for i in range(0, steps, max(1, steps // 10)):
        print("step %3d  loss %.4f" % (i + 1, losses[i]))
    print("step %3d  loss %.4f" % (steps, losses[-1]))
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 50)
