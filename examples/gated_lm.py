"""Trains a small language model data-parallel over P simulated ranks with this framework's operators.

Tokens are looked up in a table; each block is x + W2 (silu(Wg n(x)) * (Wu n(x))) with n a layer norm; a last norm and the
table itself (shared with the lookup) give the logits, and the loss is taken against the next tokens and a teacher's top
logits.  The backward pass writes every gradient into the rank's row of one flat bf16 buffer: the table's twice, first by the
output layer, then added to by the lookup's gradient.  ``zero_grad_norm`` and ``zero_adamw_step`` end the step.  Nothing waits
for the GPU but the printed loss.

    python examples/gated_lm.py [--bits 8] [--ranks 4] [--steps 100]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_shard_gb300 as z  # noqa: E402

EPS = 1e-5
TYPE, HALF = z.TYPE_BF16, torch.bfloat16


class GatedLM:
    def __init__(self, vocab: int, width: int, hidden: int, blocks: int, ranks: int, tokens: int, teacher: int = 8, bits: int = 32,
                 weight_decay: float = 0.01, temperature: float = 2.0, alpha: float = 0.5, seed: int = 0, device: str = "cuda"):
        self.v, self.d, self.h, self.blocks, self.ranks, self.tokens, self.k = vocab, width, hidden, blocks, ranks, tokens, teacher
        self.temperature, self.alpha = temperature, alpha
        # a block: the norm's weight and bias, gate and up projection (halves of one matrix), down projection
        self.shapes = [(vocab, width)] + [(width,), (width,), (2 * hidden, width), (width, hidden)] * blocks + [(width,), (width,)]
        gen = torch.Generator(device=device).manual_seed(seed)
        offsets, total = [], 0
        for s in self.shapes:
            offsets.append(total)
            total += -(-math.prod(s) // 256) * 256
        self.offsets = offsets
        self.master = torch.zeros(total, device=device)
        self.params = torch.zeros(total, dtype=HALF, device=device)
        self.grads = torch.zeros((ranks, total), dtype=HALF, device=device)
        state = torch.zeros if bits == 32 else (lambda n, device: torch.zeros(n, dtype=torch.float8_e4m3fn, device=device))
        self.m, self.v2 = state(total, device=device), state(total, device=device)
        self.m_scale, self.v_scale = (torch.zeros(total // 256, device=device) for _ in range(2))
        rows = []
        for k, (s, at) in enumerate(zip(self.shapes, offsets)):
            n = math.prod(s)
            if len(s) == 2:
                self.master[at:at + n] = torch.randn(n, generator=gen, device=device) / math.sqrt(s[1])
            elif (k - 1) % 4 == 0:
                self.master[at:at + n] = 1.0
            row = dict(grad=self.grads[0, at:], rank_stride=total, master=self.master[at:], m=self.m[at:], v=self.v2[at:], param=self.params[at:], n=n,
                       weight_decay=weight_decay if len(s) == 2 else 0.0)
            if bits == 8:
                row.update(m_scale=self.m_scale[at // 256:], v_scale=self.v_scale[at // 256:])
            rows.append(row)
        self.params.copy_(self.master)
        self.plan = z.zero_adamw_plan(rows, ranks, TYPE, TYPE, bits)
        self.stats = torch.zeros(3, device=device)
        # activations of one rank at a time; rows of the logits start on 16 bytes
        t = tokens
        new = lambda *s: torch.empty(s, dtype=HALF, device=device)  # noqa: E731
        self.x = [new(t, width) for _ in range(blocks + 1)]
        self.n = [new(t, width) for _ in range(blocks + 1)]
        self.mean, self.rstd = (torch.empty((blocks + 1, t), device=device) for _ in range(2))
        self.gu, self.a = [new(t, 2 * hidden) for _ in range(blocks)], [new(t, hidden) for _ in range(blocks)]
        self.ldl = -(-vocab // 8) * 8
        self.logits = torch.zeros((t, self.ldl), dtype=HALF, device=device)
        self.da, self.dn, self.dx = new(t, hidden), new(t, width), new(t, width)
        self.loss = torch.empty(t, device=device)
        aligned = width % 8 == 0 and hidden % 8 == 0
        need = [z.zero_linear_workspace(t, k, n, z.ACT_NONE, back, aligned) for k, n in ((hidden, width), (width, vocab)) for back in (False, True)]
        need += [z.zero_gated_workspace(t, width, hidden, back, aligned) for back in (False, True)]
        need += [z.zero_embed_workspace(t, width, vocab), z.zero_layernorm_workspace(t, width)]
        self.ws = torch.empty(max(need + [16]), dtype=torch.uint8, device=device)

    def tensor(self, flat: torch.Tensor, k: int) -> torch.Tensor:
        at, s = self.offsets[k], self.shapes[k]
        return flat[at:at + math.prod(s)].view(s)

    def _block(self, flat: torch.Tensor, b: int):
        w, bias, gu, down = (self.tensor(flat, 1 + 4 * b + k) for k in range(4))
        return w, bias, gu[:self.h], gu[self.h:], down

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        """The logits of ids [tokens] (int32; -1 is padding); keeps what the backward pass needs."""
        d, h, t, ws = self.d, self.h, self.tokens, self.ws
        table = self.tensor(self.params, 0)
        z.zero_embed_forward(ids, table, d, self.x[0], d, t, d, self.v, 1.0, TYPE)
        for b in range(self.blocks):
            w, bias, wg, wu, down = self._block(self.params, b)
            gu = self.gu[b]
            z.zero_layernorm_forward(self.x[b], d, w, bias, self.n[b], d, self.mean[b], self.rstd[b], t, d, EPS, TYPE)
            z.zero_gated_forward(self.n[b], d, wg, d, wu, d, None, None, self.a[b], h, gu, 2 * h, gu[:, h:], 2 * h, t, d, h, z.ACT_SILU, TYPE, ws, ws.numel())
            z.zero_linear_forward(self.a[b], h, down, h, None, self.x[b], d, self.x[b + 1], d, None, 0, t, h, d, z.ACT_NONE, TYPE, ws, ws.numel())
        w, bias = (self.tensor(self.params, len(self.shapes) - 2 + k) for k in range(2))
        z.zero_layernorm_forward(self.x[-1], d, w, bias, self.n[-1], d, self.mean[-1], self.rstd[-1], t, d, EPS, TYPE)
        z.zero_linear_forward(self.n[-1], d, table, d, None, None, 0, self.logits, self.ldl, None, 0, t, d, self.v, z.ACT_NONE, TYPE, ws, ws.numel())
        return self.logits[:, :self.v]

    def backward(self, ids, targets, index, teacher, rank: int, grad_scale: float) -> None:
        """The rows' losses into ``loss`` and every gradient, times grad_scale, into the rank's row."""
        d, h, t, ws, row = self.d, self.h, self.tokens, self.ws, self.grads[rank]
        # the logits become their gradient
        z.zero_distill_loss(self.logits, self.ldl, targets, index, teacher, self.k, None, self.loss, self.logits, self.ldl, t, self.v, self.k,
                            self.temperature, self.alpha, grad_scale, TYPE, z.TYPE_FP32)
        table, dtable = self.tensor(self.params, 0), self.tensor(row, 0)
        z.zero_linear_backward(self.logits, self.ldl, None, 0, self.n[-1], d, table, d, self.dn, d, dtable, d, None, t, d, self.v, z.ACT_NONE, TYPE,
                               ws, ws.numel())
        last = len(self.shapes) - 2
        z.zero_layernorm_backward(self.dn, d, self.x[-1], d, self.tensor(self.params, last), self.mean[-1], self.rstd[-1], None, 0, self.dx, d,
                                  self.tensor(row, last), self.tensor(row, last + 1), t, d, TYPE, ws, ws.numel())
        for b in reversed(range(self.blocks)):
            w, _, wg, wu, down = self._block(self.params, b)
            dw, dbias, dwg, dwu, ddown = self._block(row, b)
            gu = self.gu[b]
            z.zero_linear_backward(self.dx, d, None, 0, self.a[b], h, down, h, self.da, h, ddown, h, None, t, h, d, z.ACT_NONE, TYPE, ws, ws.numel())
            z.zero_gated_backward(self.da, h, gu, 2 * h, gu[:, h:], 2 * h, self.n[b], d, wg, d, wu, d, self.dn, d, dwg, d, dwu, d, None, None, t, d, h,
                                  z.ACT_SILU, TYPE, ws, ws.numel())
            # dx += the norm's gradient: the residual's passes by
            z.zero_layernorm_backward(self.dn, d, self.x[b], d, w, self.mean[b], self.rstd[b], self.dx, d, self.dx, d, dw, dbias, t, d, TYPE, ws, ws.numel())
        z.zero_embed_backward(ids, self.dx, d, dtable, d, t, d, self.v, 1.0, True, TYPE, ws, ws.numel())

    def step(self, batch, t: int, lr: float, max_norm: float = 1.0) -> torch.Tensor:
        """One training step on a (ids, targets, index, teacher) per rank; the ranks' mean loss (on the GPU)."""
        losses = []
        for r, (ids, targets, index, teacher) in enumerate(batch):
            self.forward(ids)
            self.backward(ids, targets, index, teacher, r, 1.0 / self.tokens)
            losses.append(self.loss.mean())
        z.zero_grad_norm(self.plan, 1.0, max_norm, self.stats)
        z.zero_adamw_step(self.plan, self.stats, t, lr, 0.9, 0.999, 1e-8, t)
        return torch.stack(losses).mean()


def data(model: GatedLM, step: int, device: str = "cuda"):
    """Per rank: tokens, each the next one's only clue (a fixed map of the vocabulary), the next tokens, and a teacher who
    knows the map."""
    gen = torch.Generator(device=device).manual_seed(1000 + step)
    out = []
    for _ in range(model.ranks):
        ids = torch.randint(0, model.v, (model.tokens,), generator=gen, device=device)
        targets = (ids * 7 + 3) % model.v
        index = (targets[:, None] + torch.arange(model.k, device=device)) % model.v
        teacher = torch.randn((model.tokens, model.k), generator=gen, device=device)
        teacher[:, 0] += 6.0
        ids[::50] = -1  # padding
        targets[::50] = -1
        out.append((ids.int(), targets.int(), index.int(), teacher))
    return out


def train(steps: int = 100, bits: int = 32, ranks: int = 4, vocab: int = 500, width: int = 128, hidden: int = 256, blocks: int = 2,
          tokens: int = 512, lr: float = 2e-3, report: int = 10) -> list:
    model = GatedLM(vocab, width, hidden, blocks, ranks, tokens, bits=bits)
    losses = []
    for t in range(1, steps + 1):
        losses.append(model.step(data(model, t), t, lr * min(1.0, t / 20)))
        if report and t % report == 0:
            print(f"step {t}: loss {float(losses[-1]):.4f}  gradient norm {float(model.stats[0]):.4f}", flush=True)
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--bits", type=int, default=32, choices=(32, 8))
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    z.build()
    train(a.steps, a.bits, a.ranks)
