"""The linear layer's gradients at the ends of their ranges: outputs of more than 2^30 columns."""
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
