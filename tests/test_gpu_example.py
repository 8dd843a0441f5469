"""examples/residual_mlp.py: the linear layers, the gradient norm and AdamW together."""
import importlib.util
import math
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    spec = importlib.util.spec_from_file_location("residual_mlp", os.path.join(ROOT, "examples", "residual_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_training(ex, steps):
    """The same training in fp32 with autograd and the AdamW formulas written out; the losses."""
    model = ex.ResidualMLP(128, 512, 2, 4, 256)
    p = [model.tensor(model.master, k).clone().requires_grad_() for k in range(len(model.shapes))]
    m, v = ([torch.zeros_like(q) for q in p] for _ in range(2))
    losses = []
    for t in range(1, steps + 1):
        x, y = ex.data(model, t)
        total = 0.0
        for r in range(4):
            h = x[r].float()
            for b in range(2):
                w1, b1, w2, b2 = p[4 * b:4 * b + 4]
                h = h + torch.nn.functional.gelu(h @ w1.T + b1, approximate="tanh") @ w2.T + b2
            total = total + ((h - y[r].float()) ** 2).mean() / 4
        grads = torch.autograd.grad(total, p)
        losses.append(float(total.detach()))
        clip = min(1.0, 1.0 / (math.sqrt(sum(float(g.square().sum()) for g in grads)) + 1e-6))
        lr = 2e-3 * min(1.0, t / 20)
        with torch.no_grad():
            for q, g, a, c in zip(p, grads, m, v):
                a.mul_(0.9).add_(g * clip, alpha=0.1)
                c.mul_(0.999).add_((g * clip) ** 2, alpha=0.001)
                if q.dim() == 2:
                    q.mul_(1 - lr * 0.01)
                q.sub_(lr * (a / (1 - 0.9 ** t)) / ((c / (1 - 0.999 ** t)).sqrt() + 1e-8))
    return losses


def test_training_follows_the_plain_form(ex):
    """120 steps with 32-bit and with 8-bit moments against the same training in plain fp32: the losses stay within 2 %
    (fp16 weights and activations, 3 bits of mantissa in the moments), and fall."""
    plain = plain_training(ex, 120)
    assert plain[-1] < 0.7 * plain[0]
    for bits in (32, 8):
        losses = ex.train(steps=120, bits=bits, report=0)
        worst = max(abs(a - b) / b for a, b in zip(losses, plain))
        assert worst < 0.02, (bits, worst)


def test_gradients_against_autograd(ex):
    """Two ranks' rows against autograd in 64 bits through the same network.  Activations and gradients between layers are
    rounded to fp16 (2^-11) a dozen times on the way; the norm of a tensor's error is within 2 % of its gradient's."""
    model = ex.ResidualMLP(width=72, hidden=200, blocks=2, ranks=2, tokens=100)
    x, y = ex.data(model, 1)
    for r in range(2):
        diff = model.forward(x[r]).float() - y[r].float()
        model.backward((diff * (2 * 256.0 / diff.numel())).half(), r)
    torch.cuda.synchronize()
    for r in range(2):
        p = [model.tensor(model.params, k).double().requires_grad_() for k in range(len(model.shapes))]
        h = x[r].double()
        for b in range(2):
            w1, b1, w2, b2 = p[4 * b:4 * b + 4]
            h = h + torch.nn.functional.gelu(h @ w1.T + b1, approximate="tanh") @ w2.T + b2
        ((h - y[r].double()) ** 2).mean().mul(256.0).backward()
        for k, q in enumerate(p):
            got = model.tensor(model.grads[r], k).double()
            assert float((got - q.grad).norm()) <= 0.02 * float(q.grad.norm()), k
