"""The linear layer's gradients at the ends of their ranges: outputs of more than 2^30 columns, infinite and NaN gradients
in places that ReLU masks."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    yield zlib
    assert zlib.zero_train_timeouts() == 0


@pytest.mark.parametrize("N,products", [(2 ** 30 + 1, False), (2 ** 31 - 513, False), (2 ** 31 - 513, True)])
def test_bias_gradient_of_very_many_columns(z, N, products):
    """More than 2^30 features, one token: its gradient is the bias's gradient (and, with one input of 1, the weight's)."""
    dy = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    for at in range(0, N, 2 ** 28):
        dy[:, at:at + 2 ** 28].normal_()
    x = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    db, dw = torch.zeros_like(dy[0]), torch.zeros_like(dy[0]) if products else None
    n = z.zero_linear_workspace(1, 1, N, 0, True, False)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_linear_backward(dy, N, None, 0, x, 1, None, 0, None, 0, dw, 1, db, 1, 1, N, 0, 1, ws, n)
    assert torch.equal(db, dy[0]) and (not products or torch.equal(dw, dy[0]))


@pytest.mark.parametrize("T,K,N,pad", [(300, 64, 264, 0), (20, 40, 56, 0), (517, 65, 71, 1), (5000, 136, 1032, 0)])
@pytest.mark.parametrize("ty", [0, 1])
def test_relu_masks_non_finite_gradients(z, T, K, N, pad, ty):
    """Where ReLU's pre-activation is not above 0 (or is NaN) its gradient is 0 whatever dy holds: infinities and NaN there
    leave the bits of the gradients as they are with 0 in their place."""
    dt = (torch.float16, torch.bfloat16)[ty]
    gen = torch.Generator(device="cuda").manual_seed(T)
    rows = lambda t, width, scale: (torch.randn((t, width + pad), generator=gen, device="cuda") * scale).to(dt)[:, :width]  # noqa: E731
    x, w, dy, pre = rows(T, K, 1.0), rows(N, K, 0.1), rows(T, N, 0.1), rows(T, N, 1.0)
    pre[0], pre[1, ::3] = 0.0, math.nan
    off = ~(pre > 0)
    pick = torch.randint(0, 40, (T, N), generator=gen, device="cuda")
    bad = torch.where(pick < 2, math.inf, torch.where(pick < 4, -math.inf, math.nan)).to(dt)
    dirty = torch.empty((T, N + pad), dtype=dt, device="cuda")[:, :N].copy_(torch.where(off & (pick < 6), bad, dy))
    clean = torch.empty((T, N + pad), dtype=dt, device="cuda")[:, :N].copy_(torch.where(off, torch.zeros_like(dy), dy))
    assert int((~torch.isfinite(dirty)).sum()) > T * N // 20
    n = z.zero_linear_workspace(T, K, N, 1, True, pad == 0)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    out = []
    for d in (dirty, clean):
        dx, dw, db = (torch.empty(s, dtype=dt, device="cuda") for s in ((T, K), (N, K), (N,)))
        z.zero_linear_backward(d, N + pad, pre, N + pad, x, K + pad, w, K + pad, dx, K, dw, K, db, T, K, N, 1, ty, ws, n)
        out.append((dx, dw, db))
    for a, b in zip(*out):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
