"""Trains a residual MLP data-parallel over P simulated ranks with this framework's operators.

Each block is x + W2 gelu(W1 x + b1) + b2.  Every rank runs its own batch forward and backward
through ``zero_linear_forward`` / ``zero_linear_backward``; the backward pass writes each weight's and
bias's gradient straight into the rank's row of one flat fp16 buffer.  Then ``zero_grad_norm`` takes
the norm of the ranks' mean gradient over all tensors (undoing the loss scale) and
``zero_adamw_step`` reads the P rows, averages, clips and updates every tensor in one launch, with
fp32 or 8-bit moments.  Nothing waits for the GPU but the printed loss.

    python examples/residual_mlp.py [--bits 8] [--ranks 4] [--steps 200]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_shard_gb300 as z  # noqa: E402


class ResidualMLP:
    def __init__(self, width: int, hidden: int, blocks: int, ranks: int, tokens: int, bits: int = 32,
                 weight_decay: float = 0.01, seed: int = 0, device: str = "cuda"):
        self.d, self.h, self.blocks, self.ranks, self.tokens = width, hidden, blocks, ranks, tokens
        shapes = [(hidden, width), (hidden,), (width, hidden), (width,)] * blocks
        gen = torch.Generator(device=device).manual_seed(seed)
        half = dict(dtype=torch.float16, device=device)
        # every tensor starts on a multiple of 256 elements of the flat buffers: whole vectors, and blocks of 8-bit scales
        offsets, total = [], 0
        for s in shapes:
            offsets.append(total)
            total += -(-math.prod(s) // 256) * 256
        self.master = torch.zeros(total, device=device)
        self.params = torch.zeros(total, **half)
        self.grads = torch.zeros((ranks, total), **half)
        state = torch.zeros if bits == 32 else (lambda n, device: torch.zeros(n, dtype=torch.float8_e4m3fn, device=device))
        self.m, self.v = state(total, device=device), state(total, device=device)
        self.m_scale, self.v_scale = (torch.zeros(total // 256, device=device) for _ in range(2))
        tensors = []
        for k, (s, at) in enumerate(zip(shapes, offsets)):
            n = math.prod(s)
            if len(s) == 2:
                scale = 1 / math.sqrt(s[1]) * (0.5 if k % 4 == 2 else 1.0)
                self.master[at:at + n] = torch.randn(n, generator=gen, device=device) * scale
            t = dict(grad=self.grads[0, at:], rank_stride=total, master=self.master[at:], m=self.m[at:], v=self.v[at:],
                     param=self.params[at:], n=n, weight_decay=weight_decay if len(s) == 2 else 0.0)
            if bits == 8:
                t.update(m_scale=self.m_scale[at // 256:], v_scale=self.v_scale[at // 256:])
            tensors.append(t)
        self.params.copy_(self.master)
        self.offsets, self.shapes = offsets, shapes
        self.plan = z.zero_adamw_plan(tensors, ranks, z.TYPE_FP16, z.TYPE_FP16, bits)
        self.stats = torch.zeros(3, device=device)
        # activations of one rank at a time, and the layers' workspace
        t = tokens
        self.x = [torch.empty((t, width), **half) for _ in range(blocks + 1)]
        self.z = [torch.empty((t, hidden), **half) for _ in range(blocks)]
        self.a = [torch.empty((t, hidden), **half) for _ in range(blocks)]
        self.da, self.dx = torch.empty((t, hidden), **half), torch.empty((t, width), **half)
        aligned = width % 8 == 0 and hidden % 8 == 0
        need = max(z.zero_linear_workspace(t, k, n, z.ACT_GELU, back, aligned) for k, n in ((width, hidden), (hidden, width))
                   for back in (False, True))
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)

    def tensor(self, flat: torch.Tensor, k: int) -> torch.Tensor:
        at, s = self.offsets[k], self.shapes[k]
        return flat[at:at + math.prod(s)].view(s)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """The output for x [tokens, width]; keeps what the backward pass needs."""
        d, h, t, ws = self.d, self.h, self.tokens, self.ws
        self.x[0].copy_(x)
        for b in range(self.blocks):
            w1, b1, w2, b2 = (self.tensor(self.params, 4 * b + k) for k in range(4))
            z.zero_linear_forward(self.x[b], d, w1, d, b1, None, 0, self.a[b], h, self.z[b], h, t, d, h, z.ACT_GELU,
                                  z.TYPE_FP16, ws, ws.numel())
            z.zero_linear_forward(self.a[b], h, w2, h, b2, self.x[b], d, self.x[b + 1], d, None, 0, t, h, d, z.ACT_NONE,
                                  z.TYPE_FP16, ws, ws.numel())
        return self.x[-1]

    def backward(self, dy: torch.Tensor, rank: int) -> None:
        """Gradients of every weight and bias into the rank's row, from dy [tokens, width] of the last forward."""
        d, h, t, ws = self.d, self.h, self.tokens, self.ws
        row = self.grads[rank]
        for b in reversed(range(self.blocks)):
            w1, _, w2, _ = (self.tensor(self.params, 4 * b + k) for k in range(4))
            g = [self.tensor(row, 4 * b + k) for k in range(4)]
            z.zero_linear_backward(dy, d, None, 0, self.a[b], h, w2, h, self.da, h, g[2], h, g[3], t, h, d, z.ACT_NONE,
                                   z.TYPE_FP16, ws, ws.numel())
            z.zero_linear_backward(self.da, h, self.z[b], h, self.x[b], d, w1, d, self.dx, d, g[0], d, g[1], t, d, h,
                                   z.ACT_GELU, z.TYPE_FP16, ws, ws.numel())
            dy = dy + self.dx  # the residual's gradient is dy itself

    def step(self, batch, targets, t: int, lr: float, loss_scale: float = 1024.0, max_norm: float = 1.0) -> torch.Tensor:
        """One training step on batch and targets [ranks, tokens, width]; the ranks' mean loss (on the GPU)."""
        losses = []
        for r in range(self.ranks):
            diff = self.forward(batch[r]).float() - targets[r].float()
            losses.append(diff.square().mean())
            self.backward((diff * (2 * loss_scale / diff.numel())).half(), r)
        z.zero_grad_norm(self.plan, 1.0 / loss_scale, max_norm, self.stats)
        z.zero_adamw_step(self.plan, self.stats, t, lr, 0.9, 0.999, 1e-8, t)
        return torch.stack(losses).mean()


def data(model: ResidualMLP, step: int, device: str = "cuda"):
    """A fixed smooth map to learn, on fresh inputs."""
    gen = torch.Generator(device=device).manual_seed(1000 + step)
    x = torch.randn((model.ranks, model.tokens, model.d), generator=gen, device=device)
    return x.half(), (x + torch.sin(2 * x.roll(1, -1))).half()


def train(steps: int = 200, bits: int = 32, ranks: int = 4, width: int = 128, hidden: int = 512, blocks: int = 2,
          tokens: int = 256, lr: float = 2e-3, report: int = 20) -> list:
    model = ResidualMLP(width, hidden, blocks, ranks, tokens, bits)
    losses = []
    for t in range(1, steps + 1):
        losses.append(model.step(*data(model, t), t, lr * min(1.0, t / 20)))
        if report and t % report == 0:
            print(f"step {t}: loss {float(losses[-1]):.4f}  gradient norm {float(model.stats[0]):.4f}", flush=True)
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--bits", type=int, default=32, choices=(32, 8))
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    z.build()
    train(a.steps, a.bits, a.ranks)
