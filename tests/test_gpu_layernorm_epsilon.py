"""Layer norm with an epsilon as large as fp32 has, beside variances below, near and above it.

Tolerances: those of test_gpu_layernorm_mean.py (c times the mean of the centred values' magnitudes for what is left of the mean,
2c + 2^-21 of the statistics)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, assert_within  # noqa: E402
from test_gpu_layernorm_mean import chain, forward, z  # noqa: E402,F401


@pytest.mark.parametrize("eps", [1.0, 1e30, 2e37, 3e37, 1e38, 3.4e38])
@pytest.mark.parametrize("D", [24, 60, 333, 2048, 9000, 20000])
@pytest.mark.parametrize("ty", [0, 1])
def test_large_epsilon(z, eps, D, ty):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((7, D), generator=gen, device="cuda")
    for k, scale in enumerate((1.0, 1e18, 4e18, 1e19, 2e19, 1e36, 0.0)):
        x[k] *= scale if ty else min(scale, 1e4)
    x = x.to(DT[ty])
    w = torch.randn(D, generator=gen, device="cuda").to(DT[ty])
    y, mean, rstd = forward(z, x, w, None, eps, ty)
    xd, wd = x.double(), w.double()
    m = xd.mean(1, keepdim=True)
    d = xd - m
    s = ((d ** 2).mean(1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32))) ** -0.5
    h = d * s
    c = chain(D)
    e = (c + 2.0 ** -24) * xd.abs().mean(1, keepdim=True)
    left = c * (d.abs().mean(1, keepdim=True) + e)
    es = 2 * c + 2.0 ** -21
    ref = h * wd
    err = (left * s + h.abs() * es + 2.0 ** -22 * (xd.abs() + e) * s) * wd.abs() + 2.0 ** -23 * ref.abs()
    assert bool(((rstd.double() / s[:, 0] - 1).abs() <= es).all()), (rstd.double() / s[:, 0] - 1).tolist()
    assert bool(((mean.double() - m[:, 0]).abs() <= (left + e)[:, 0]).all())
    tiny = 2.0 ** -133 if ty else 0.0                          # half of bf16's last step
    assert_within(y, ref, err + tiny, ty)
