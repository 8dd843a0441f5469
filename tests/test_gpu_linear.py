"""The linear layer with bias, activation and residual, and its gradients, against the formulas in 64 bits.

Tolerances.  Products of 16-bit operands are exact in fp32; a sum of K of them in fp32, rounded towards zero at
worst at each step, is off by at most (K + 8) 2^-23 times the sum of their magnitudes.  The activations' derivatives
are at most 1.13 in magnitude and their evaluation is off by a few fp32 ulp of |z| + 1 (2^-18 covers the fast
exponential and quotient).  A result in 16 bits is rounded once, by at most u of itself (2^-8 for bf16, 2^-11 for
fp16, whose subnormals are 2^-24 apart); dz is rounded once before the products of the backward pass."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {0: torch.float16, 1: torch.bfloat16}
HALF_ULP = {0: 2.0 ** -11, 1: 2.0 ** -8}
SUB = {0: 2.0 ** -25, 1: 0.0}
NAN = float("nan")


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    yield zlib
    assert zlib.zero_train_timeouts() == 0


def act64(a, z):
    if a == 1:
        return torch.where(z < 0, torch.zeros_like(z), z)     # NaN stays NaN
    if a == 2:
        return torch.nn.functional.gelu(z, approximate="tanh")
    if a == 3:
        return z * torch.sigmoid(z)
    return z


def slope64(a, z):
    if a == 0:
        return torch.ones_like(z)
    if a == 1:
        return (z > 0).double()
    if a == 2:
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s + z * s * (1 - s)


def rows(t, width, pad, dt, gen, scale=1.0, shift=0):
    """[t, width] values in rows of width + pad elements, `shift` elements into their buffer; NaN around them."""
    buf = torch.full((t * (width + pad) + shift + 16,), NAN, dtype=dt, device="cuda")
    v = torch.as_strided(buf, (t, width), (width + pad, 1), shift)
    v.copy_(torch.randn((t, width), generator=gen, device="cuda") * scale)
    return v, buf


def outside_untouched(view, buf):
    keep = buf.clone()
    torch.as_strided(keep, view.shape, view.stride(), view.storage_offset()).fill_(NAN)
    return bool(torch.isnan(keep).all()) and not bool(torch.isnan(view).any())


def workspace(z, T, K, N, act, backward, aligned):
    n = z.zero_linear_workspace(T, K, N, act, backward, aligned)
    return torch.full((max(n, 16),), 0x7F, dtype=torch.uint8, device="cuda"), n


def check_forward(z, T, K, N, act, ty, pad=0, shift=0, bias=True, res=True, keep=True, inplace=False, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, u = DT[ty], HALF_ULP[ty]
    x, _ = rows(T, K, pad, dt, gen, 1.0, shift)
    w, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    b = torch.randn(N + 1, generator=gen, device="cuda").to(dt)[shift % 2:][:N] if bias else None
    r, _ = rows(T, N, pad, dt, gen, 1.0, shift) if res else (None, None)
    y, ybuf = rows(T, N, pad, dt, gen, 0.0, shift)
    if inplace:
        y.copy_(r)
        want_r, r = r, y
    else:
        want_r = r
    zz, zbuf = rows(T, N, pad, dt, gen, 0.0, shift) if keep else (None, None)
    ws, n = workspace(z, T, K, N, act, False, pad % 8 == 0 and K % 8 == 0 and shift % 8 == 0)
    z.zero_linear_forward(x, K + pad, w, K + pad, b, r, N + pad, y, N + pad, zz, N + pad, T, K, N, act, ty, ws, n)
    torch.cuda.synchronize()
    xd, wd = x.double(), w.double()
    zd, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    if b is not None:
        zd, mag = zd + b.double(), mag + b.double().abs()
    ez = (K + 8) * 2.0 ** -23 * mag + 2.0 ** -40
    yd = act64(act, zd)
    ey = 1.13 * ez + (2.0 ** -18 * (zd.abs() + 1) if act else 0)
    if res:
        yd = yd + want_r.double()
        ey = ey + 2.0 ** -23 * yd.abs()
    assert bool(((y.double() - yd).abs() <= ey + u * (yd.abs() + ey) + SUB[ty]).all()), float((y.double() - yd).abs().max())
    assert outside_untouched(y, ybuf)
    if keep:
        assert bool(((zz.double() - zd).abs() <= ez + u * (zd.abs() + ez) + SUB[ty]).all())
        assert outside_untouched(zz, zbuf)


def check_backward(z, T, K, N, act, ty, pad=0, shift=0, want=("dx", "dw", "db"), seed=0, dwpad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, u = DT[ty], HALF_ULP[ty]
    x, _ = rows(T, K, pad, dt, gen, 1.0, shift)
    w, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    dy, _ = rows(T, N, pad, dt, gen, 0.5, shift)
    zz, _ = rows(T, N, pad, dt, gen, 1.0, shift)
    if act == 1:
        zz[0, :] = 0                                      # ReLU's derivative at 0 is 0
    dx, dxb = rows(T, K, pad, dt, gen, 0.0, shift)
    dw, dwb = rows(N, K, dwpad, dt, gen, 0.0, shift)
    db, dbb = rows(1, N, 0, dt, gen, 0.0, shift)
    ws, n = workspace(z, T, K, N, act, True, pad % 8 == 0 and K % 8 == 0 and N % 8 == 0 and shift % 8 == 0)
    z.zero_linear_backward(dy, N + pad, zz if act else None, N + pad, x, K + pad, w, K + pad,
                           dx if "dx" in want else None, K + pad, dw if "dw" in want else None, K + dwpad,
                           db if "db" in want else None, T, K, N, act, ty, ws, n)
    torch.cuda.synchronize()
    dyd, xd, wd = dy.double(), x.double(), w.double()
    s = slope64(act, zz.double())
    dz = dyd * s
    ezf = dyd.abs() * 2.0 ** -18 * (zz.double().abs() + 1) if act else torch.zeros_like(dz)  # dz in fp32
    ez = ezf + (u * (dz.abs() + ezf) + SUB[ty] if act else 0)                                   # and rounded
    for name, got, buf, ref, mag, err, terms in (
            ("dx", dx, dxb, dz @ wd, (dz.abs() + ez) @ wd.abs(), ez @ wd.abs(), N),
            ("dw", dw, dwb, dz.T @ xd, (dz.abs() + ez).T @ xd.abs(), ez.T @ xd.abs(), T),
            ("db", db, dbb, dz.sum(0, keepdim=True), (dz.abs() + ezf).sum(0, keepdim=True), ezf.sum(0, keepdim=True), T)):
        if name not in want:
            assert not bool(got.any())
            continue
        e = err + (terms + 8) * 2.0 ** -23 * mag
        bad = (got.double() - ref).abs() - (e + u * (ref.abs() + e) + SUB[ty])
        assert float(bad.max()) <= 0, (name, float(bad.max()), float((got.double() - ref).abs().max()))
        assert outside_untouched(got, buf), name


# few tokens (the operands change sides), one column width each, then tiles with the contraction cut or not
FORWARD = [(1, 64, 128), (1, 1, 1), (2, 65, 7), (4, 512, 1000), (16, 100, 128), (17, 63, 129), (33, 1000, 255), (64, 192, 257),
           (65, 128, 64), (128, 4096, 136), (100, 2048, 2000), (129, 64, 8), (200, 65, 100), (256, 1024, 256), (300, 1000, 520),
           (1000, 3000, 70), (511, 8, 513)]


@pytest.mark.parametrize("T,K,N", FORWARD)
@pytest.mark.parametrize("act,ty,pad,shift", [(0, 0, 0, 0), (1, 1, 8, 0), (2, 1, 0, 0), (3, 0, 3, 1), (2, 0, 0, 8)])
def test_forward(z, T, K, N, act, ty, pad, shift):
    check_forward(z, T, K, N, act, ty, pad, shift, seed=T + N)


MANY = [(5000, 200, 1000, 0), (4993, 1000, 1100, 8), (6000, 72, 1027, 0), (2500, 520, 2600, 3), (20000, 64, 256, 0), (4096, 2048, 2050, 0)]
# few tokens against wide layers: contractions cut over a cluster
WIDE = [(5, 2048, 4096), (30, 2048, 2048), (60, 2048, 2000), (128, 2048, 4096), (250, 2048, 2048), (200, 200, 9000), (400, 320, 4096), (2048, 1024, 1024), (512, 2048, 2048)]


@pytest.mark.parametrize("T,K,N,pad", MANY)
@pytest.mark.parametrize("act,ty", [(0, 1), (2, 0), (3, 1)])
def test_forward_many_tiles(z, T, K, N, pad, act, ty):
    check_forward(z, T, K, N, act, ty, pad, seed=K)


def test_every_kernel_is_covered(z):
    """The shapes of the tests above and below reach every kernel: each tile width, whole and cut contractions, pairs,
    one product and two in a launch, two launches."""
    seen, both = set(), set()
    for T, K, N in FORWARD + [s[:3] for s in MANY] + WIDE:
        p = z.zero_linear_plan(T, K, N, 0)
        seen.add((p["rows"], p["columns"], p["per_sm"], p["cluster"] > 1))
    for T, K, N in BACKWARD + [s[:3] for s in MANY_BACK]:
        p = z.zero_linear_plan(T, K, N, 3)
        both.add((p["rows"], p["columns"], p["per_sm"], p["launches"]))
    for want in [(128, 16, 2, False), (128, 16, 2, True), (128, 32, 2, True), (128, 64, 1, True), (128, 64, 2, False),
                 (128, 128, 1, False), (128, 128, 1, True), (256, 256, 1, True)]:
        assert want in seen, (want, sorted(seen))
    assert {(r, c) for r, c, _, n in both if n == 1} >= {(128, 64), (128, 128), (256, 256)}, sorted(both)
    assert any(n == 2 for *_, n in both), sorted(both)


@pytest.mark.parametrize("T,K,N", WIDE)
def test_forward_wide(z, T, K, N):
    check_forward(z, T, K, N, 2, 1, 0, 0, seed=T)
    check_forward(z, T, K, N, 0, 0, 2, 0, seed=T)              # rows on 4 bytes


@pytest.mark.parametrize("bias,res,keep,inplace", [(False, False, False, False), (True, False, False, False), (False, True, False, False),
                                                   (False, False, True, False), (True, True, True, True)])
@pytest.mark.parametrize("T,K,N", [(3, 200, 300), (300, 200, 304), (5000, 100, 1000)])
def test_optional_parts(z, T, K, N, bias, res, keep, inplace):
    check_forward(z, T, K, N, 2, 1, 0, 0, bias, res, keep, inplace)


BACKWARD = [(1, 64, 128), (1, 1, 1), (3, 65, 7), (16, 200, 128), (100, 1000, 257), (128, 136, 4096), (129, 64, 64), (200, 65, 100),
            (300, 520, 1000), (4096, 64, 48), (511, 513, 8), (10000, 130, 100)]


@pytest.mark.parametrize("T,K,N", BACKWARD)
@pytest.mark.parametrize("act,ty,pad,shift,dwpad", [(0, 0, 0, 0, 0), (1, 1, 8, 0, 8), (2, 1, 0, 0, 0), (3, 0, 3, 1, 5), (0, 1, 1, 0, 0), (2, 0, 0, 8, 0)])
def test_backward(z, T, K, N, act, ty, pad, shift, dwpad):
    check_backward(z, T, K, N, act, ty, pad, shift, seed=T + K, dwpad=dwpad)


MANY_BACK = [(5000, 1000, 200, 0), (300, 1000, 5000, 0), (5100, 1030, 5000, 0), (2600, 2500, 523, 3), (4, 2048, 8192, 0), (60, 2048, 2048, 0), (512, 784, 1192, 0)]


@pytest.mark.parametrize("T,K,N,pad", MANY_BACK)
@pytest.mark.parametrize("act,ty", [(0, 1), (2, 0)])
def test_backward_many_tiles(z, T, K, N, pad, act, ty):
    check_backward(z, T, K, N, act, ty, pad, seed=K)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")])
@pytest.mark.parametrize("act", [0, 2])
def test_backward_parts(z, want, act):
    check_backward(z, 200, 136, 264, act, 1, want=want)
    check_backward(z, 20, 135, 263, act, 1, pad=1, want=want)


def test_gradients_against_differences(z):
    """Central differences of sum(c * y) in 64 bits, y by the formula, against the kernel's dx, dw and db.  The
    difference quotient with step h is off by h^2/6 times the third derivative (below 16 |c| for these values)."""
    T, K, N, h = 5, 12, 9, 1e-4
    gen = torch.Generator(device="cuda").manual_seed(0)
    for act in (0, 2, 3):
        x, w = (torch.randn((n, K), generator=gen, device="cuda").half() * 0.5 for n in (T, N))
        b, c = torch.randn(N, generator=gen, device="cuda").half(), torch.randn((T, N), generator=gen, device="cuda").half()
        loss = lambda x, w, b: (c.double() * act64(act, x @ w.T + b)).sum()  # noqa: E731
        zz, y = torch.empty_like(c), torch.empty_like(c)
        ws, n = workspace(z, T, K, N, act, True, False)
        z.zero_linear_forward(x, K, w, K, b, None, 0, y, N, zz, N, T, K, N, act, 0, ws, n)
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        z.zero_linear_backward(c, N, zz, N, x, K, w, K, dx, K, dw, K, db, T, K, N, act, 0, ws, n)
        args = [x.double(), w.double(), b.double()]
        for k, got in enumerate((dx, dw, db)):
            flat = args[k].view(-1)
            for i in range(0, flat.numel(), 7):
                keep = float(flat[i])
                flat[i] = keep + h
                up = loss(*args)
                flat[i] = keep - h
                down = loss(*args)
                flat[i] = keep
                want = float((up - down) / (2 * h))
                # z is stored in fp16 (its slope moves by at most 1.1 of that), dz and the result are rounded once each
                terms = float(c.double().abs().sum()) * 3
                assert abs(float(got.view(-1)[i]) - want) <= 4 * 2.0 ** -11 * terms + 1e-6


def test_no_tokens(z):
    K, N = 24, 40
    w = torch.randn((N, K), device="cuda").half()
    dw, db = torch.full((N, K + 8), NAN, dtype=torch.float16, device="cuda"), torch.full((N,), NAN, dtype=torch.float16, device="cuda")
    y = torch.full((8,), 5.0, dtype=torch.float16, device="cuda")
    z.zero_linear_forward(None, K, w, K, None, None, 0, y, N, None, 0, 0, K, N, 2, 0)
    z.zero_linear_backward(None, N, None, N, None, K, w, K, None, K, dw, K + 8, db, 0, K, N, 2, 0)
    torch.cuda.synchronize()
    assert bool((y == 5).all()) and not dw[:, :K].any() and bool(torch.isnan(dw[:, K:]).all()) and not db.any()


def test_non_finite_values_stay_in_their_rows(z):
    """A NaN token and an infinite one leave every other token's row alone."""
    for T, K, N in ((8, 100, 200), (300, 100, 200), (5000, 100, 1000)):
        x = torch.randn((T, K), device="cuda").bfloat16()
        w = torch.randn((N, K), device="cuda").bfloat16()
        y0, y1 = (torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ws, n = workspace(z, T, K, N, 0, False, False)
        z.zero_linear_forward(x, K, w, K, None, None, 0, y0, N, None, 0, T, K, N, 0, 1, ws, n)
        x[1, 3], x[5, 7] = NAN, math.inf
        z.zero_linear_forward(x, K, w, K, None, None, 0, y1, N, None, 0, T, K, N, 0, 1, ws, n)
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[1] = ok[5] = False
        assert torch.equal(y0[ok], y1[ok]) and bool(torch.isnan(y1[1]).all()) and not bool(torch.isfinite(y1[5]).any())


def test_activations_at_extreme_values(z):
    """Pre-activations as far out as bf16 goes, through a layer of one input (z = x): the activation and its slope take
    their limits, NaN stays NaN."""
    vals = [0.0, -0.0, 1e-38, -1e-38, 30.0, -30.0, 1e4, -1e4, 1e19, -1e19, 3e38, -3e38, math.inf, NAN]
    T = len(vals)
    x = torch.tensor(vals, device="cuda").bfloat16()[:, None]
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    ws, n = workspace(z, T, 1, 1, 2, True, False)
    for act in (1, 2, 3):
        y, zz, dx = (torch.empty((T, 1), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        z.zero_linear_forward(x, 1, one, 1, None, None, 0, y, 1, zz, 1, T, 1, 1, act, 1, ws, n)
        z.zero_linear_backward(one.expand(T, 1).contiguous(), 1, zz, 1, x, 1, one, 1, dx, 1, None, 0, None, T, 1, 1, act, 1, ws, n)
        xd = x.double()
        want = torch.where(xd > 40, xd, torch.where(xd < -40, torch.zeros_like(xd), act64(act, xd)))
        slope = torch.where(xd > 40, 1.0, torch.where(xd < -40, 0.0, slope64(act, xd)))
        if act == 1:
            slope[-1] = 0                                     # the slope of ReLU is a comparison
        for got, ref in ((y, want), (dx, slope)):
            got, ref = got.double(), ref.double()
            assert torch.equal(torch.isnan(got), torch.isnan(ref)), (act, got, ref)
            ok = ~torch.isnan(ref) & ~torch.isinf(ref)
            assert bool((got[ok] - ref[ok]).abs().le(2.0 ** -7 * ref[ok].abs() + 1e-30).all()), (act, got, ref)
            assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])


def test_large_offsets(z):
    """An output of more than 2^31 elements, few inputs: its first and last rows."""
    T, K, N = 270000, 64, 8192
    x, w = torch.randn((T, K), device="cuda").bfloat16(), (torch.randn((N, K), device="cuda") / 8).bfloat16()
    b = torch.randn(N, device="cuda").bfloat16()
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    z.zero_linear_forward(x, K, w, K, b, None, 0, y, N, None, 0, T, K, N, 1, 1)
    rowsel = torch.cat([torch.arange(300), torch.arange(262140, 262150), torch.arange(T - 300, T)]).cuda()
    ref = (x[rowsel].double() @ w.double().T + b.double()).clamp(min=0)
    mag = x[rowsel].double().abs() @ w.double().abs().T + b.double().abs()
    assert bool(((y[rowsel].double() - ref).abs() <= (K + 8) * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs() + 1e-30).all())
    dw, db = torch.empty_like(w), torch.empty_like(b)
    ws, n = workspace(z, T, K, N, 1, True, True)
    dy = y                                                     # any values will do: y as its own gradient, ReLU by y's sign
    z.zero_linear_backward(dy, N, y, N, x, K, None, 0, None, 0, dw, K, db, T, K, N, 1, 1, ws, n)
    part = [(dy[r:r + 30000].float(), x[r:r + 30000].float()) for r in range(0, T, 30000)]
    ref = sum((d.double().sum(0) for d, _ in part))
    assert bool(((db.double() - ref).abs() <= (T + 8) * 2.0 ** -23 * ref + 2.0 ** -8 * ref).all())
    cols = torch.arange(0, N, 1000, device="cuda")
    ref = sum(d[:, cols].double().T @ v.double() for d, v in part)
    mag = sum(d[:, cols].double().T @ v.double().abs() for d, v in part)
    assert bool(((dw[cols].double() - ref).abs() <= (T + 8) * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs()).all())


def test_column_slices_of_one_buffer_and_streams(z):
    """x, the residual and y as column slices of one buffer; the same bits on another stream and from a graph."""
    T, K, N = 200, 64, 96
    buf = torch.randn((T, K + N + N), device="cuda").half()
    w = torch.randn((N, K), device="cuda").half()
    ld = buf.shape[1]
    x, r, y = buf[:, :K], buf[:, K:K + N], buf[:, K + N:]
    z.zero_linear_forward(x, ld, w, K, None, r, ld, y, ld, None, 0, T, K, N, 3, 0)
    zd = x.double() @ w.double().T
    want = act64(3, zd) + r.double()
    assert bool(((y.double() - want).abs() <= 2.0 ** -10 * (want.abs() + zd.abs() + 1)).all())
    first = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        z.zero_linear_forward(x, ld, w, K, None, r, ld, y, ld, None, 0, T, K, N, 3, 0, stream=side)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, y)


def test_gradients_into_a_ranks_slice(z):
    """dw and db written into odd places of the flat gradient vector of one rank."""
    T, K, N, P = 70, 31, 45, 2
    g = torch.full((P, 5000), NAN, dtype=torch.float16, device="cuda")
    x, w, dy = (torch.randn(s, device="cuda").half() * 0.3 for s in ((T, K), (N, K), (T, N)))
    ws, n = workspace(z, T, K, N, 0, True, False)
    at = 333
    z.zero_linear_backward(dy, N, None, 0, x, K, w, K, None, 0, g[1, at:], K, g[1, at + N * K:], T, K, N, 0, 0, ws, n)
    torch.cuda.synchronize()
    ref = torch.cat([(dy.double().T @ x.double()).view(-1), dy.double().sum(0)])
    got = g[1, at:at + N * K + N].double()
    assert bool(((got - ref).abs() <= 2.0 ** -11 * ref.abs() + (T + 8) * 2.0 ** -23 * 0.3 * 0.3 * T * 16 + 2.0 ** -25).all())
    assert bool(torch.isnan(g[0]).all()) and bool(torch.isnan(g[1, :at]).all()) and bool(torch.isnan(g[1, at + N * K + N:]).all())


def test_refused_calls_write_nothing(z):
    T, K, N = 16, 32, 48
    x, w = torch.randn((T, K), device="cuda").half(), torch.randn((N, K), device="cuda").half()
    y = torch.full((T, N), 3.0, dtype=torch.float16, device="cuda")
    good = dict(x=x, ldx=K, w=w, ldw=K, bias=None, res=None, ldr=0, y=y, ldy=N, zz=None, ldz=0, T=T, K=K, N=N, act=0, ty=0, ws=None, n=0)
    E, A, O = z.ZERO_EINVAL, z.ZERO_EALIGN, z.ZERO_EOVERLAP
    for kw, code in [(dict(x=None), E), (dict(w=None), E), (dict(y=None), E), (dict(T=-1), E), (dict(K=0), E), (dict(N=0), E), (dict(ldx=K - 1), E),
                     (dict(ldy=N - 1), E), (dict(act=4), E), (dict(ty=2), E), (dict(y=y.data_ptr() + 1), A), (dict(y=x, ldy=N), O),
                     (dict(zz=y, ldz=N), O), (dict(res=y.data_ptr() + 2, ldr=N), O), (dict(K=K - 1, ldx=K - 1, ldw=K - 1), E)]:
        a = dict(good, **kw)
        with pytest.raises(z.ZeroError) as e:
            z.zero_linear_forward(a["x"], a["ldx"], a["w"], a["ldw"], a["bias"], a["res"], a["ldr"], a["y"], a["ldy"], a["zz"], a["ldz"],
                                  a["T"], a["K"], a["N"], a["act"], a["ty"], a["ws"], a["n"])
        assert e.value.code == code, kw
    torch.cuda.synchronize()
    assert bool((y == 3).all())
