"""Layer norm and its gradients against the formulas in 64 bits.

Tolerances.  A thread adds at most n values of a row before the threads' sums are joined (n = 64, more only for rows above
16384), so a row's sum in fp32 is off by at most c = (n + 60) 2^-24 times the sum of magnitudes.  With m the mean of |x|, the
mean is off by c m; the centred squares' mean by a factor of 1 + 2c + 2^-22 and (c m)^2; so y is off by (c m s + |h| (2c + 2^-21)
+ 2^-22 (|x| + |mean|) s) |w| + 2^-23 |b|, with one rounding more.  The backward pass takes the statistics as they are: h is off by
2^-23 (|x| + |mean|) s, the rows' sums by c, the columns' sums by (rows + 64) 2^-24 of the sum of magnitudes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, NAN, assert_within, outside_untouched, replayed, rows  # noqa: E402


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def chain(D):
    return (max(64, D // 1024 + 8) + 60) * 2.0 ** -24


def vector(D, dt, gen, scale, offset, shift):
    return (torch.randn(D + 8, generator=gen, device="cuda") * scale + offset).to(dt)[shift % 8:][:D]


def check_forward(z, T, D, ty, pad=0, shift=0, weight=True, bias=True, stats=True, inplace=False, eps=1e-5, offset=0.3, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    dt = DT[ty]
    x, xbuf = rows(T, D, pad, dt, gen, scale, shift, offset)
    w = vector(D, dt, gen, 0.2, 1.0, shift) if weight else None
    b = vector(D, dt, gen, 0.2, 0.0, shift) if bias else None
    y, buf = (x, xbuf) if inplace else rows(T, D, pad, dt, gen, 0.0, shift)
    xd = x.double()
    mean, rstd = (torch.full((T + 2,), NAN, device="cuda") if stats else None for _ in range(2))
    z.zero_layernorm_forward(x, D + pad, w, b, y, D + pad, mean, rstd, T, D, eps, ty)
    torch.cuda.synchronize()
    c = chain(D)
    m = xd.mean(1, keepdim=True)
    var = ((xd - m) ** 2).mean(1, keepdim=True)
    s = (var + eps) ** -0.5
    h = (xd - m) * s
    em = c * xd.abs().mean(1, keepdim=True) + 2.0 ** -24 * m.abs()
    es = (2 * c + 2.0 ** -21 + em ** 2 / (var + eps))          # relative
    wd = w.double() if weight else torch.ones(D, dtype=torch.float64, device="cuda")
    ref = h * wd + (b.double() if bias else 0)
    err = (em * s + h.abs() * es + 2.0 ** -22 * (xd.abs() + m.abs()) * s) * wd.abs() + 2.0 ** -23 * ref.abs()
    assert_within(y, ref, err, ty)
    assert outside_untouched(y, buf)
    if stats:
        assert bool(((mean[:T].double() - m[:, 0]).abs() <= em[:, 0]).all())
        assert bool(((rstd[:T].double() / s[:, 0] - 1).abs() <= es[:, 0]).all())
        assert bool(torch.isnan(mean[T:]).all()) and bool(torch.isnan(rstd[T:]).all())


WIDTHS = [1, 7, 8, 64, 255, 256, 264, 513, 1000, 1024, 1032, 2048, 2049, 4096, 5000, 8192, 8200, 12289, 16384, 16392, 40000]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [1, 9, 130])
@pytest.mark.parametrize("ty,pad,shift", [(0, 0, 0), (1, 8, 0), (1, 0, 8), (0, 3, 1), (1, 1, 0)])
def test_forward(z, T, D, ty, pad, shift):
    check_forward(z, T, D, ty, pad, shift)


@pytest.mark.parametrize("weight,bias,stats,inplace", [(False, False, True, False), (True, False, False, False), (False, True, True, True), (True, True, False, True)])
@pytest.mark.parametrize("T,D", [(5, 200), (70, 1001), (20, 2048), (3, 20000)])
def test_forward_parts(z, weight, bias, stats, inplace, T, D):
    check_forward(z, T, D, 1, 0, 0, weight, bias, stats, inplace)


def test_rows_far_from_zero(z):
    """Values whose mean is far above their spread: the variance is not lost in a difference."""
    check_forward(z, 50, 1000, 0, offset=1000.0, scale=4.0)
    check_forward(z, 50, 3000, 1, offset=-64.0, scale=2.0)
    check_forward(z, 10, 600, 1, eps=1e-30, offset=0.0, scale=1e-12)


def test_values_as_large_as_bf16_has(z):
    """Squares above fp32's range: the statistics of rows of up to 3e38, constant ones and ordinary ones among them."""
    big = torch.finfo(torch.bfloat16).max
    for D in (24, 333, 2048, 20000):
        x = torch.randn((6, D), device="cuda").to(DT[1])
        x[1] *= 1e30
        x[2], x[2, ::2] = big, -big
        x[3] = big
        x[4] *= 2e19
        y = torch.empty_like(x)
        mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        z.zero_layernorm_forward(x, D, None, None, y, D, mean, rstd, 6, D, 1e-5, 1)
        xd = x.double()
        m = xd.mean(1, keepdim=True)
        s = (((xd - m) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
        ref = (xd - m) * s
        ref[3], s[3] = ref[3] * 0, 1e-5 ** -0.5
        keep = torch.ones(6, dtype=torch.bool, device="cuda")
        keep[3] = False
        # rstd of the largest rows is below the normal range: 20 bits of it are left
        assert_within(y[keep], ref[keep], 2.0 ** -15 * (ref[keep].abs() + 1), 1)
        assert bool(torch.isfinite(y[3]).all())
        assert bool(((rstd.double() / s[:, 0] - 1).abs()[keep] < 2.0 ** -15).all())
        # their gradients
        dy = torch.randn((6, D), device="cuda").to(DT[1])
        dx = torch.empty_like(x)
        z.zero_layernorm_backward(dy, D, x, D, None, mean, rstd, None, 0, dx, D, None, None, 6, D, 1)
        r = rstd.double()[:, None]
        h = (xd - mean.double()[:, None]) * r
        a = dy.double()
        want = r * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
        assert bool(((dx.double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * r * (1 + h.abs()) * 4 + 1e-40)[keep].all())


def check_backward(z, T, D, ty, pad=0, shift=0, res=True, weight=True, want=("dx", "dw", "db"), inplace=None):
    gen = torch.Generator(device="cuda").manual_seed(T + D + 1)
    dt = DT[ty]
    x, _ = rows(T, D, pad, dt, gen, 1.5, shift, 0.4)
    dy, dybuf = rows(T, D, pad, dt, gen, 0.5, shift)
    r, rbuf = rows(T, D, pad, dt, gen, 0.5, shift) if res else (None, None)
    w = vector(D, dt, gen, 0.2, 1.0, shift) if weight else None
    xd, dyd, rd = x.double(), dy.double(), r.double() if res else 0
    mean = xd.mean(1).float()
    rstd = (((xd - xd.mean(1, keepdim=True)) ** 2).mean(1) + 1e-5).rsqrt().float()
    dx, buf = {"dy": (dy, dybuf), "res": (r, rbuf), None: (None, None)}[inplace]
    if dx is None:
        dx, buf = rows(T, D, pad, dt, gen, 0.0, shift)
    dw, db = (vector(D, dt, gen, 0.0, 0.0, shift) for _ in range(2))
    n = z.zero_layernorm_workspace(T, D)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    z.zero_layernorm_backward(dy, D + pad, x, D + pad, w, mean, rstd, r, D + pad, dx if "dx" in want else None, D + pad,
                              dw if "dw" in want else None, db if "db" in want else None, T, D, ty, ws, n)
    torch.cuda.synchronize()
    c = chain(D)
    m, s = mean.double()[:, None], rstd.double()[:, None]
    h = (xd - m) * s
    H = (xd.abs() + m.abs()) * s                              # h is off by 2^-23 of it
    a = dyd * (w.double() if weight else 1)
    c1 = (a * h).mean(1, keepdim=True)
    ref = s * (a - a.mean(1, keepdim=True) - h * c1) + rd
    err = s * (2.0 ** -22 * a.abs() + 2 * c * a.abs().mean(1, keepdim=True) + H.abs() * 2.0 ** -22 * c1.abs()
               + h.abs() * (2 * c + 2.0 ** -22) * (a.abs() * H).mean(1, keepdim=True)) + 2.0 ** -22 * ref.abs() + 2.0 ** -23 * (rd.abs() if res else 0)
    for name, got, want_, e in (("dx", dx, ref, err), ("dw", dw, (dyd * h).sum(0), (T + 64) * 2.0 ** -23 * (dyd.abs() * H).sum(0)),
                                ("db", db, dyd.sum(0), (T + 64) * 2.0 ** -24 * dyd.abs().sum(0))):
        if name in want:
            assert_within(got, want_, e, ty, name)
        elif inplace is None:
            assert not bool(got.any())
    assert outside_untouched(dx, buf)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [1, 9, 130])
@pytest.mark.parametrize("ty,pad,shift", [(0, 0, 0), (1, 8, 0), (1, 0, 8), (0, 3, 1), (1, 1, 0)])
def test_backward(z, T, D, ty, pad, shift):
    check_backward(z, T, D, ty, pad, shift)


@pytest.mark.parametrize("T,D", [(5000, 100), (3001, 331), (2600, 2048), (4000, 1000), (700, 4096), (650, 9000), (320, 17000)])
@pytest.mark.parametrize("ty", [0, 1])
def test_backward_many_rows(z, T, D, ty):
    check_backward(z, T, D, ty)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "dw"), ("dw", "db")])
@pytest.mark.parametrize("res,weight", [(True, False), (False, True)])
@pytest.mark.parametrize("T,D", [(40, 201), (100, 2048), (70, 9000)])
def test_backward_parts(z, want, res, weight, T, D):
    check_backward(z, T, D, 1, 0, 0, res, weight, want)


@pytest.mark.parametrize("inplace,T,D", [("dy", 100, 333), ("res", 100, 333), ("dy", 50, 2048), ("res", 50, 8192), ("res", 20, 9001), ("dy", 20, 16000), ("res", 10, 17001), ("dy", 1000, 64)])
def test_backward_in_place(z, inplace, T, D):
    check_backward(z, T, D, 0, inplace=inplace)


def test_gradients_against_differences(z):
    """Central differences of sum(c * y) in 64 bits, y by the formula: step h is off by h^2/6 times the third derivative
    (below 100 |c| here), and the kernel's gradients by their roundings."""
    T, D, h = 3, 20, 1e-4
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, c = (torch.randn((T, D), generator=gen, device="cuda").half() for _ in range(2))
    w, b = torch.randn(D, generator=gen, device="cuda").half(), torch.randn(D, generator=gen, device="cuda").half()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n = z.zero_layernorm_workspace(T, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_layernorm_forward(x, D, w, b, y, D, mean, rstd, T, D, 1e-3, 0)
    z.zero_layernorm_backward(c, D, x, D, w, mean, rstd, None, 0, dx, D, dw, db, T, D, 0, ws, n)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        return (c.double() * ((x - m) * (((x - m) ** 2).mean(1, keepdim=True) + 1e-3) ** -0.5 * w + b)).sum()

    args = [x.double(), w.double(), b.double()]
    terms = float(c.double().abs().sum())
    for k, got in enumerate((dx, dw, db)):
        flat = args[k].view(-1)
        for i in range(0, flat.numel(), 3):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss(*args)
            flat[i] = keep - h
            down = loss(*args)
            flat[i] = keep
            assert abs(float(got.view(-1)[i]) - float((up - down) / (2 * h))) <= 2.0 ** -11 * abs(float(got.view(-1)[i])) + 2.0 ** -18 * terms + 100 * h * h * terms


def test_no_rows_and_foreign_rows(z):
    D = 72
    dw, db = (torch.full((D + 8,), NAN, dtype=torch.float16, device="cuda") for _ in range(2))
    z.zero_layernorm_forward(None, D, None, None, None, D, None, None, 0, D, 1e-5, 0)
    z.zero_layernorm_backward(None, D, None, D, None, None, None, None, 0, None, D, dw, db, 0, D, 0)
    torch.cuda.synchronize()
    assert not dw[:D].any() and not db[:D].any() and bool(torch.isnan(dw[D:]).all()) and bool(torch.isnan(db[D:]).all())
    # a NaN row and an infinite one leave the others' outputs alone
    for T, D in ((40, 72), (40, 2048), (40, 333)):
        x = torch.randn((T, D), device="cuda").to(DT[1])
        y = [torch.empty_like(x) for _ in range(2)]
        z.zero_layernorm_forward(x, D, None, None, y[0], D, None, None, T, D, 1e-5, 1)
        x[3, 1], x[7, 2] = NAN, float("inf")
        z.zero_layernorm_forward(x, D, None, None, y[1], D, None, None, T, D, 1e-5, 1)
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[3] = ok[7] = False
        assert torch.equal(y[0][ok], y[1][ok]) and bool(torch.isnan(y[1][3]).all()) and bool(torch.isnan(y[1][7]).all())


def test_graph_repeats_the_bits(z):
    T, D = 1500, 328
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = rows(T, D, 0, DT[1], gen)[0], rows(T, D, 0, DT[1], gen)[0]
    w, b = vector(D, DT[1], gen, 0.2, 1.0, 0), vector(D, DT[1], gen, 0.2, 0.0, 0)
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")]
    y, dx, dw, db, mean, rstd = outs
    n = z.zero_layernorm_workspace(T, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(stream=None):
        z.zero_layernorm_forward(x, D, w, b, y, D, mean, rstd, T, D, 1e-5, 1, stream=stream)
        z.zero_layernorm_backward(dy, D, x, D, w, mean, rstd, y, D, dx, D, dw, db, T, D, 1, ws, n, stream=stream)

    call()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    assert all(torch.equal(p, q) for p, q in zip(first, replayed(call, outs)))


def test_large_offsets(z):
    """Matrices of more than 2^31 elements: their first and last rows."""
    T, D = 2 ** 21 + 300, 1032
    x = torch.zeros((T, D), dtype=DT[1], device="cuda")
    some = torch.cat([torch.arange(100), torch.arange(T - 300, T)]).cuda()
    x[some] = torch.randn((len(some), D), device="cuda").to(DT[1])
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    keep = x[some].double()
    z.zero_layernorm_forward(x, D, None, None, x, D, mean, rstd, T, D, 1e-5, 1)
    m = keep.mean(1, keepdim=True)
    ref = (keep - m) * (((keep - m) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
    assert_within(x[some], ref, 2.0 ** -16 * (ref.abs() + 1), 1)
    dx = torch.empty_like(x)
    z.zero_layernorm_backward(x, D, x, D, None, mean, rstd, None, 0, dx, D, None, None, T, D, 1)
    a, r = x[some].double(), rstd[some].double()[:, None]
    h = (a - mean[some].double()[:, None]) * r
    want = r * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    assert_within(dx[some], want, 2.0 ** -15 * r * (a.abs() + h.abs() + 1) * (1 + h.abs().mean(1, keepdim=True)), 1)
