"""Layer norm of rows whose mean is far above their spread, constant rows among them, against the formulas in 64 bits.

Tolerances.  With c as in test_gpu_layernorm.py (a row's sum in fp32 is off by at most c times the sum of magnitudes), the mean's
first value is off by at most e = c |m| + 2^-24 |m|, but the centred values' own mean is taken out of them again: what is left is c
times the mean of the centred values' magnitudes, which is at most |x - m| on average plus e.  So y is off by
c (mean|x - m| + e) s, |h| (2c + 2^-21) for the statistics, and 2^-23 (|x - m| + e) s for the two roundings of a centred value;
the saved mean by those c (mean|x - m| + e) and its own rounding, 2^-24 |m|.  rstd is off by 2c + 2^-21 of itself, and by what
rounding leaves of (e s)^2, 4c of it.

Constant rows whose sum has at most 24 significant bits: every partial sum is exact, so is the mean, and y is the bias."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, assert_within, rows  # noqa: E402


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def chain(D):
    return (max(64, D // 1024 + 8) + 60) * 2.0 ** -24


def forward(z, x, w, b, eps, ty, ld=None):
    T, D = x.shape
    y = torch.empty((T, D), dtype=x.dtype, device="cuda")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    z.zero_layernorm_forward(x, ld or D, w, b, y, D, mean, rstd, T, D, eps, ty)
    torch.cuda.synchronize()
    return y, mean, rstd


@pytest.mark.parametrize("value,D,ty", [(1000.0, 1001, 0), (60000.0, 2000, 0), (3000.0, 768, 0), (3008.0, 768, 1), (1000.0, 333, 1), (-7.0, 3, 0), (65504.0, 7, 1),
                                        (-60000.0, 201, 0), (2.0 ** 100, 5000, 1), (1e-3, 100, 1), (1000.0, 12000, 0), (1.5, 16384, 1), (24.0, 40000, 1), (1000.0, 16392, 1)])
@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_constant_rows_are_the_bias(z, value, D, ty, eps):
    v = torch.full((1,), value).to(DT[ty])
    m, exponent = torch.frexp(v.double())
    assert float(m.abs() * 2 ** (11 if ty == 0 else 8) % 1) == 0
    units = int(m.abs() * 2 ** 11)
    while units % 2 == 0:
        units //= 2
    assert units * D < 2 ** 24                                 # every partial sum is exact
    gen = torch.Generator(device="cuda").manual_seed(D)
    for T in (1, 70):
        x = v.cuda().expand(T, D).contiguous()
        w, b = (torch.randn(D, generator=gen, device="cuda").to(DT[ty]) for _ in range(2))
        y, mean, rstd = forward(z, x, w, b, eps, ty)
        assert torch.equal(y, b.expand(T, D)), float((y.double() - b.double()).abs().max())
        assert bool((mean.double() == float(v)).all())
        e = float(torch.tensor(eps, dtype=torch.float32))
        assert bool(((rstd.double() * e ** 0.5 - 1).abs() <= 2.0 ** -22).all())


@pytest.mark.parametrize("T,D", [(5, 24), (70, 333), (40, 1001), (300, 2000), (20, 4104), (9, 12001), (6, 16384), (3, 50000)])
@pytest.mark.parametrize("ty,pad,shift", [(0, 0, 0), (1, 8, 0), (0, 3, 1)])
@pytest.mark.parametrize("offset,scale", [(1000.0, 0.0), (-50000.0, 40.0), (3000.0, 3.0), (0.37, 1e-3)])
def test_rows_far_from_zero(z, T, D, ty, pad, shift, offset, scale):
    """Constant rows (scale 0), and rows of a few neighbouring 16-bit values."""
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    x, _ = rows(T, D, pad, DT[ty], gen, scale, shift, offset)
    x[T // 2] = offset
    x[T // 2, D // 2] = x[T // 2, D // 2] * 1.01                # one value beside all others
    w, b = (torch.randn(D, generator=gen, device="cuda").to(DT[ty]) for _ in range(2))
    eps = 1e-5
    y, mean, rstd = forward(z, x, w, b, eps, ty, D + pad)
    xd, wd, bd = x.double(), w.double(), b.double()
    m = xd.mean(1, keepdim=True)
    d = xd - m
    s = ((d ** 2).mean(1, keepdim=True) + eps) ** -0.5
    h = d * s
    c = chain(D)
    e = (c + 2.0 ** -24) * m.abs()
    left = c * (d.abs().mean(1, keepdim=True) + e)
    es = 2 * c + 2.0 ** -21 + 4 * c * (e * s) ** 2
    ref = h * wd + bd
    err = (left * s + h.abs() * es + 2.0 ** -23 * (d.abs() + e) * s) * wd.abs() + 2.0 ** -23 * (ref.abs() + bd.abs())
    assert_within(y, ref, err, ty)
    assert bool(((mean.double() - m[:, 0]).abs() <= (left + 2.0 ** -24 * m.abs())[:, 0]).all())
    assert bool(((rstd.double() / s[:, 0] - 1).abs() <= es[:, 0]).all())


@pytest.mark.parametrize("T,D,ty", [(40, 1001, 0), (300, 2000, 0), (50, 768, 1), (9, 12001, 0), (3, 20000, 0)])
def test_gradients_of_constant_rows(z, T, D, ty):
    """h is 0 in a constant row, so that dx = (a - mean(a)) / sqrt(eps), and the weight's gradient is 0."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.full((T, D), 1000.0, device="cuda").to(DT[ty])
    dy, _ = rows(T, D, 0, DT[ty], gen, 2.0 ** -8)
    w = torch.randn(D, generator=gen, device="cuda").to(DT[ty])
    eps = 1e-3
    _, mean, rstd = forward(z, x, w, None, eps, ty)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    n = z.zero_layernorm_workspace(T, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_layernorm_backward(dy, D, x, D, w, mean, rstd, None, 0, dx, D, dw, db, T, D, ty, ws, n)
    torch.cuda.synchronize()
    a = dy.double() * w.double()
    s = float(torch.tensor(eps, dtype=torch.float32)) ** -0.5
    ref = s * (a - a.mean(1, keepdim=True))
    assert_within(dx, ref, 2.0 ** -21 * s * a.abs() + 2 * chain(D) * s * a.abs().mean(1, keepdim=True) + 2.0 ** -21 * ref.abs(), ty)
    assert not bool(dw.any())
