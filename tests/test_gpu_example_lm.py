"""examples/gated_lm.py: embedding, layer norm, gated projections, linear layers, the loss, the gradient norm and AdamW together."""
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
    spec = importlib.util.spec_from_file_location("gated_lm", os.path.join(ROOT, "examples", "gated_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def loss64(model, p, ids, targets, index, teacher):
    """The mean of the rows' losses in 64 bits, from tensors in the model's order."""
    there = ids >= 0
    x = torch.where(there[:, None], p[0][ids.long().clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda"))
    norm = lambda x, w, b: torch.nn.functional.layer_norm(x, (x.shape[1],), w, b, 1e-5)  # noqa: E731
    for b in range(model.blocks):
        w, bias, gu, down = p[1 + 4 * b:5 + 4 * b]
        n = norm(x, w, bias)
        g, u = n @ gu[:model.h].T, n @ gu[model.h:].T
        x = x + (torch.nn.functional.silu(g) * u) @ down.T
    s = norm(x, p[-2], p[-1]) @ p[0].T
    hard = torch.nn.functional.cross_entropy(s, targets.long(), ignore_index=-1, reduction="none")
    lp = torch.log_softmax(teacher.double() / model.temperature, 1)
    lq = torch.log_softmax(s / model.temperature, 1).gather(1, index.long())
    soft = model.temperature ** 2 * (lp.exp() * (lp - lq)).sum(1)
    return ((1 - model.alpha) * hard + model.alpha * soft).mean()


@pytest.mark.parametrize("vocab,width,hidden", [(303, 72, 200), (257, 65, 99)])
def test_gradients_against_autograd(ex, vocab, width, hidden):
    """Two ranks' rows against autograd in 64 bits through the same network.  Activations and gradients between the layers are
    rounded to bf16 (2^-8) some twenty times on the way; the norm of a tensor's error is within 5 % of its gradient's."""
    model = ex.GatedLM(vocab, width, hidden, blocks=2, ranks=2, tokens=100)
    for r, (ids, targets, index, teacher) in enumerate(ex.data(model, 1)):
        model.forward(ids)
        model.backward(ids, targets, index, teacher, r, 1.0 / model.tokens)
        torch.cuda.synchronize()
        p = [model.tensor(model.params, k).double().requires_grad_() for k in range(len(model.shapes))]
        want = loss64(model, p, ids, targets, index, teacher)
        want.backward()
        assert abs(float(model.loss.double().mean() - want.detach())) <= 0.02 * float(want.detach())
        for k, q in enumerate(p):
            got = model.tensor(model.grads[r], k).double()
            assert float((got - q.grad).norm()) <= 0.05 * float(q.grad.norm()), (r, k)


@pytest.mark.parametrize("bits", [32, 8])
def test_training_runs(ex, bits):
    """Steps of training end with finite losses and weights that moved, and repeat bit for bit."""
    runs = [ex.train(steps=5, bits=bits, ranks=2, report=0) for _ in range(2)]
    assert runs[0] == runs[1] and all(math.isfinite(x) for x in runs[0]) and len(set(runs[0])) == 5


def test_a_step_from_a_graph(ex, zlib):
    """Forward, loss and backward of a rank captured and replayed: the same gradients as eagerly."""
    model = ex.GatedLM(300, 64, 128, blocks=2, ranks=1, tokens=160)
    batch = ex.data(model, 3)[0]
    model.forward(batch[0])
    model.backward(*batch, 0, 1.0)
    torch.cuda.synchronize()
    first = model.grads.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        model.forward(batch[0])
        model.backward(*batch, 0, 1.0)
    for _ in range(2):
        model.grads.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(model.grads, first)
    assert zlib.zero_train_timeouts() == 0
