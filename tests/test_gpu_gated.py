"""The gated feed-forward projections and their gradients against the formulas in 64 bits.

Tolerances.  Products of 16-bit operands are exact in fp32; a sum of K of them in fp32, rounded towards zero at worst at each
step, is off by at most (K + 8) 2^-23 times the sum of their magnitudes (eg, eu for g and u).  The activations' slopes are at
most 1.13 in magnitude, and activation and slope are off by 2^-18 (|g| + 1) (fast exponential and quotient), so h is off by
(1.13 eg + 2^-18 (|g| + 1)) (|u| + eu) + |act(g)| eu.  A result is rounded once, by half a step; dg and du once before the products."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, HALF_ULP, NAN, SUB, assert_within, outside_untouched, replayed, rows  # noqa: E402


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    yield zlib
    assert zlib.zero_train_timeouts() == 0


def act64(a, z):
    if a == 1:
        return torch.where(z < 0, torch.zeros_like(z), z)
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


def vector(n, dt, gen, shift):
    return torch.randn(n + 8, generator=gen, device="cuda").to(dt)[shift % 8:][:n]


def workspace(z, T, K, N, backward, aligned):
    n = z.zero_gated_workspace(T, K, N, backward, aligned)
    return torch.full((max(n, 16),), 0x7F, dtype=torch.uint8, device="cuda"), n


def check_forward(z, T, K, N, act, ty, pad=0, shift=0, bias=True, keep=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[ty]
    x, _ = rows(T, K, pad, dt, gen, 1.0, shift)
    wg, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    wu, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    bg, bu = (vector(N, dt, gen, shift) if bias else None for _ in range(2))
    h, hbuf = rows(T, N, pad, dt, gen, 0.0, shift)
    g, gbuf = rows(T, N, pad, dt, gen, 0.0, shift) if keep else (None, None)
    u, ubuf = rows(T, N, pad, dt, gen, 0.0, shift) if keep else (None, None)
    ws, n = workspace(z, T, K, N, False, pad % 8 == 0 and K % 8 == 0 and shift % 8 == 0)
    z.zero_gated_forward(x, K + pad, wg, K + pad, wu, K + pad, bg, bu, h, N + pad, g, N + pad, u, N + pad, T, K, N, act, ty, ws, n)
    torch.cuda.synchronize()
    xd = x.double()
    gd, ud = xd @ wg.double().T, xd @ wu.double().T
    mg, mu = xd.abs() @ wg.double().abs().T, xd.abs() @ wu.double().abs().T
    if bias:
        gd, ud, mg, mu = gd + bg.double(), ud + bu.double(), mg + bg.double().abs(), mu + bu.double().abs()
    eg, eu = ((K + 8) * 2.0 ** -23 * m + 2.0 ** -40 for m in (mg, mu))
    a = act64(act, gd)
    ea = 1.13 * eg + (2.0 ** -18 * (gd.abs() + 1) if act > 1 else 0)
    assert_within(h, a * ud, ea * (ud.abs() + eu) + a.abs() * eu + 2.0 ** -23 * (a * ud).abs(), ty, "h")
    assert outside_untouched(h, hbuf)
    if keep:
        assert_within(g, gd, eg, ty, "g")
        assert_within(u, ud, eu, ty, "u")
        assert outside_untouched(g, gbuf) and outside_untouched(u, ubuf)


FORWARD = [(1, 64, 128), (1, 1, 1), (2, 65, 7), (4, 512, 1000), (16, 100, 64), (17, 63, 129), (33, 1000, 255), (64, 192, 257),
           (65, 128, 64), (128, 4096, 136), (100, 2048, 2000), (129, 64, 8), (129, 200, 3), (200, 65, 100), (256, 1024, 256), (300, 1000, 520),
           (1000, 3000, 70), (511, 8, 513)]


@pytest.mark.parametrize("T,K,N", FORWARD)
@pytest.mark.parametrize("act,ty,pad,shift", [(0, 0, 0, 0), (1, 1, 8, 0), (2, 1, 0, 0), (3, 0, 3, 1), (2, 0, 0, 8), (3, 1, 2, 0)])
def test_forward(z, T, K, N, act, ty, pad, shift):
    check_forward(z, T, K, N, act, ty, pad, shift, seed=T + N)


MANY = [(5000, 200, 500, 0), (4993, 1000, 555, 8), (6000, 72, 1027, 0), (2500, 520, 1300, 3), (20000, 64, 256, 0), (4096, 1024, 2050, 0), (3000, 256, 1600, 0)]
WIDE = [(5, 2048, 4096), (30, 2048, 2048), (60, 2048, 2000), (128, 2048, 4096), (250, 2048, 2048), (200, 200, 9000), (400, 320, 4096), (1024, 1024, 1024), (512, 2048, 1024), (2048, 512, 512), (2000, 512, 500)]


@pytest.mark.parametrize("T,K,N,pad", MANY)
@pytest.mark.parametrize("act,ty,keep", [(0, 1, True), (2, 0, False), (3, 1, True)])
def test_forward_many_tiles(z, T, K, N, pad, act, ty, keep):
    check_forward(z, T, K, N, act, ty, pad, seed=K, keep=keep)


@pytest.mark.parametrize("T,K,N", WIDE)
def test_forward_wide(z, T, K, N):
    check_forward(z, T, K, N, 3, 1, 0, 0, seed=T)
    check_forward(z, T, K, N, 0, 0, 2, 0, seed=T, keep=False)


@pytest.mark.parametrize("bias,keep", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T,K,N", [(3, 200, 300), (300, 200, 304), (5000, 100, 1000)])
def test_optional_parts(z, bias, keep, T, K, N):
    check_forward(z, T, K, N, 3, 1, 0, 0, bias, keep)


def check_backward(z, T, K, N, act, ty, pad=0, shift=0, want=("dx", "dwg", "dwu", "dbg", "dbu"), seed=0, dwpad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, half = DT[ty], HALF_ULP[ty]
    x, _ = rows(T, K, pad, dt, gen, 1.0, shift)
    wg, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    wu, _ = rows(N, K, pad, dt, gen, 1.0 / math.sqrt(K), shift)
    dh, _ = rows(T, N, pad, dt, gen, 0.5, shift)
    g, _ = rows(T, N, pad, dt, gen, 1.0, shift)
    u, _ = rows(T, N, pad, dt, gen, 1.0, shift)
    if act == 1:
        g[0, :] = 0                                       # ReLU's derivative at 0 is 0
    out = {"dx": rows(T, K, pad, dt, gen, 0.0, shift), "dwg": rows(N, K, dwpad, dt, gen, 0.0, shift), "dwu": rows(N, K, dwpad, dt, gen, 0.0, shift),
           "dbg": rows(1, N, 0, dt, gen, 0.0, shift), "dbu": rows(1, N, 0, dt, gen, 0.0, shift)}
    ws, n = workspace(z, T, K, N, True, pad % 8 == 0 and K % 8 == 0 and shift % 8 == 0)
    arg = {k: v[0] if k in want else None for k, v in out.items()}
    z.zero_gated_backward(dh, N + pad, g, N + pad, u, N + pad, x, K + pad, wg, K + pad, wu, K + pad, arg["dx"], K + pad, arg["dwg"], K + dwpad, arg["dwu"],
                          K + dwpad, arg["dbg"], arg["dbu"], T, K, N, act, ty, ws, n)
    torch.cuda.synchronize()
    xd, wgd, wud, dhd, gd, ud = (v.double() for v in (x, wg, wu, dh, g, u))
    du, dg = dhd * act64(act, gd), dhd * ud * slope64(act, gd)
    e = 2.0 ** -18 * (gd.abs() + 1) if act > 1 else 0
    fu, fg = dhd.abs() * e + 2.0 ** -23 * du.abs(), (dhd * ud).abs() * e + 2.0 ** -22 * dg.abs()   # in fp32
    ru, rg = (f + half * (d.abs() + f) + SUB[ty] for f, d in ((fu, du), (fg, dg)))                     # and rounded

    def product(d, r, m, terms):
        return d @ m, r @ m.abs() + (terms + 8) * 2.0 ** -23 * ((d.abs() + r) @ m.abs())

    a, b = product(dg, rg, wgd, 2 * N), product(du, ru, wud, 2 * N)
    ref = {"dx": (a[0] + b[0], a[1] + b[1]), "dwg": product(dg.T, rg.T, xd, T), "dwu": product(du.T, ru.T, xd, T)}
    for k, d, f in (("dbg", dg, fg), ("dbu", du, fu)):
        ref[k] = d.sum(0, keepdim=True), f.sum(0, keepdim=True) + (T + 8) * 2.0 ** -23 * (d.abs() + f).sum(0, keepdim=True)
    for k, (got, buf) in out.items():
        if k in want:
            assert_within(got, ref[k][0], ref[k][1], ty, k)
        else:
            assert not bool(got.any()), k
        assert outside_untouched(got, buf), k


BACKWARD = [(1, 64, 128), (1, 1, 1), (3, 65, 7), (16, 200, 128), (100, 1000, 257), (128, 136, 2048), (129, 64, 64), (200, 65, 100),
            (300, 520, 1000), (4096, 64, 48), (511, 513, 8), (10000, 130, 100)]


@pytest.mark.parametrize("T,K,N", BACKWARD)
@pytest.mark.parametrize("act,ty,pad,shift,dwpad", [(0, 0, 0, 0, 0), (1, 1, 8, 0, 8), (2, 1, 0, 0, 0), (3, 0, 3, 1, 5), (0, 1, 1, 0, 0), (3, 0, 0, 8, 0)])
def test_backward(z, T, K, N, act, ty, pad, shift, dwpad):
    check_backward(z, T, K, N, act, ty, pad, shift, seed=T + K, dwpad=dwpad)


MANY_BACK = [(5000, 1000, 200, 0), (300, 1000, 2500, 0), (5100, 1030, 2500, 0), (2600, 2500, 523, 3), (4, 2048, 4096, 0), (60, 2048, 2048, 0), (512, 784, 1192, 0)]


@pytest.mark.parametrize("T,K,N,pad", MANY_BACK)
@pytest.mark.parametrize("act,ty", [(0, 1), (3, 0)])
def test_backward_many_tiles(z, T, K, N, pad, act, ty):
    check_backward(z, T, K, N, act, ty, pad, seed=K)


@pytest.mark.parametrize("want", [("dx",), ("dwg",), ("dwu",), ("dbg",), ("dx", "dbu"), ("dwg", "dwu"), ("dwu", "dbg"), ("dx", "dwu")])
@pytest.mark.parametrize("act", [0, 3])
def test_backward_parts(z, want, act):
    check_backward(z, 200, 136, 264, act, 1, want=want)
    check_backward(z, 20, 135, 263, act, 1, pad=1, want=want)


def test_every_kernel_is_covered(z):
    """The shapes of these tests reach every kernel: each tile width, whole and cut contractions, pairs, one and two launches."""
    seen, both = set(), set()
    for T, K, N in FORWARD + [s[:3] for s in MANY] + WIDE:
        p = z.zero_gated_plan(T, K, N, 0)
        seen.add((p["rows"], p["columns"], p["per_sm"], p["cluster"] > 1))
    for T, K, N in BACKWARD + [s[:3] for s in MANY_BACK]:
        p = z.zero_gated_plan(T, K, N, 3)
        both.add((p["rows"], p["columns"], p["launches"]))
    for want in [(128, 16, 2), (128, 32, 2), (128, 64, 1), (128, 64, 2), (128, 128, 1), (256, 256, 1)]:
        assert want in {s[:3] for s in seen}, (want, sorted(seen))
    assert {s[3] for s in seen if s[0] == 128} == {True, False}, sorted(seen)
    assert {(r, c) for r, c, n in both if n == 1} >= {(128, 64), (128, 128), (256, 256)}, sorted(both)
    assert any(n == 2 for *_, n in both), sorted(both)


def test_gradients_against_differences(z):
    """Central differences of sum(c * h) in 64 bits against the kernel's gradients; step d is off by d^2/6 times the third
    derivative (below 200 |c| for these values), g, u, dg, du and the results are rounded to fp16."""
    T, K, N, d = 4, 10, 7, 1e-4
    gen = torch.Generator(device="cuda").manual_seed(0)
    for act in (0, 2, 3):
        x, wg, wu = (torch.randn((n, K), generator=gen, device="cuda").half() * 0.5 for n in (T, N, N))
        bg, bu = (torch.randn(N, generator=gen, device="cuda").half() for _ in range(2))
        c = torch.randn((T, N), generator=gen, device="cuda").half()
        h, g, u = (torch.empty_like(c) for _ in range(3))
        ws, n = workspace(z, T, K, N, True, False)
        z.zero_gated_forward(x, K, wg, K, wu, K, bg, bu, h, N, g, N, u, N, T, K, N, act, 0, ws, n)
        grads = [torch.empty_like(v) for v in (x, wg, wu, bg, bu)]
        z.zero_gated_backward(c, N, g, N, u, N, x, K, wg, K, wu, K, grads[0], K, grads[1], K, grads[2], K, grads[3], grads[4], T, K, N, act, 0, ws, n)
        loss = lambda x, wg, wu, bg, bu: (c.double() * act64(act, x @ wg.T + bg) * (x @ wu.T + bu)).sum()  # noqa: E731
        args = [v.double() for v in (x, wg, wu, bg, bu)]
        terms = float((c.double().abs() * (1 + g.double().abs()) * (1 + u.double().abs())).sum()) * 3
        for k, got in enumerate(grads):
            flat = args[k].view(-1)
            for i in range(0, flat.numel(), 5):
                keep = float(flat[i])
                flat[i] = keep + d
                up = loss(*args)
                flat[i] = keep - d
                down = loss(*args)
                flat[i] = keep
                assert abs(float(got.view(-1)[i]) - float((up - down) / (2 * d))) <= 4 * 2.0 ** -11 * terms + 200 * d * d * terms, (act, k, i)


def test_no_tokens(z):
    K, N = 24, 40
    w = torch.randn((2 * N, K), device="cuda").half()
    dw = torch.full((2 * N, K + 8), NAN, dtype=torch.float16, device="cuda")
    db = torch.full((2 * N + 1,), NAN, dtype=torch.float16, device="cuda")
    z.zero_gated_forward(None, K, w, K, w[N:], K, None, None, None, N, None, 0, None, 0, 0, K, N, 3, 0)
    z.zero_gated_backward(None, N, None, N, None, N, None, K, w, K, w[N:], K, None, K, dw, K + 8, dw[N:], K + 8, db, db[N:], 0, K, N, 3, 0)
    torch.cuda.synchronize()
    assert not dw[:, :K].any() and bool(torch.isnan(dw[:, K:]).all()) and not db[:2 * N].any() and bool(torch.isnan(db[2 * N]))


def test_one_matrix_for_both_weights_and_graph(z):
    """Weights, kept values and weight gradients as halves of one matrix each; the same bits from a replayed graph."""
    for T, K, N in ((5, 72, 104), (300, 128, 200), (4000, 136, 520)):
        gen = torch.Generator(device="cuda").manual_seed(T)
        x, w, dh = rows(T, K, 0, DT[1], gen)[0], rows(2 * N, K, 0, DT[1], gen, K ** -0.5)[0], rows(T, N, 0, DT[1], gen)[0]
        h, gu = torch.empty((T, N), dtype=DT[1], device="cuda"), torch.empty((T, 2 * N), dtype=DT[1], device="cuda")
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * N, dtype=DT[1], device="cuda")
        ws, n = workspace(z, T, K, N, True, True)
        outs = [h, gu, dx, dw, db]

        def call(stream=None):
            z.zero_gated_forward(x, K, w, K, w[N:], K, None, None, h, N, gu, 2 * N, gu[:, N:], 2 * N, T, K, N, 3, 1, ws, n, stream=stream)
            z.zero_gated_backward(dh, N, gu, 2 * N, gu[:, N:], 2 * N, x, K, w, K, w[N:], K, dx, K, dw, K, dw[N:], K, db, db[N:], T, K, N, 3, 1, ws, n, stream=stream)

        call()
        torch.cuda.synchronize()
        first = [o.clone() for o in outs]
        gd, ud = (x.double() @ w.double().T).split(N, 1)
        ref = act64(3, gd) * ud
        assert bool(((h.double() - ref).abs() <= 2.0 ** -7 * (ref.abs() + 0.01 * (1 + gd.abs()) * (1 + ud.abs()))).all())
        assert all(torch.equal(p, q) for p, q in zip(first, replayed(call, outs)))


def test_non_finite_values_stay_in_their_rows(z):
    for T, K, N in ((8, 100, 200), (300, 100, 200), (5000, 100, 1000)):
        x, wg, wu = (torch.randn((n, K), device="cuda").to(DT[1]) for n in (T, N, N))
        h = [torch.empty((T, N), dtype=DT[1], device="cuda") for _ in range(2)]
        ws, n = workspace(z, T, K, N, False, False)
        z.zero_gated_forward(x, K, wg, K, wu, K, None, None, h[0], N, None, 0, None, 0, T, K, N, 0, 1, ws, n)
        x[1, 3], x[5, 7] = NAN, math.inf
        z.zero_gated_forward(x, K, wg, K, wu, K, None, None, h[1], N, None, 0, None, 0, T, K, N, 0, 1, ws, n)
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[1] = ok[5] = False
        assert torch.equal(h[0][ok], h[1][ok]) and bool(torch.isnan(h[1][1]).all()) and not bool(torch.isfinite(h[1][5]).any())


def test_large_offsets(z):
    """Outputs of more than 2^31 elements, few inputs: their first and last rows, and the weights' gradients."""
    T, K, N = 270000, 64, 8192
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, _ = rows(T, K, 0, DT[1], gen)
    wg, wu = rows(N, K, 0, DT[1], gen, 0.125)[0], rows(N, K, 0, DT[1], gen, 0.125)[0]
    h, g, u = (torch.empty((T, N), dtype=DT[1], device="cuda") for _ in range(3))
    z.zero_gated_forward(x, K, wg, K, wu, K, None, None, h, N, g, N, u, N, T, K, N, 1, 1)
    some = torch.cat([torch.arange(200), torch.arange(262140, 262150), torch.arange(T - 300, T)]).cuda()
    xs = x[some].double()
    gd, ud = xs @ wg.double().T, xs @ wu.double().T
    eg, eu = ((K + 8) * 2.0 ** -23 * (xs.abs() @ w.double().abs().T) for w in (wg, wu))
    assert_within(g[some], gd, eg, 1)
    assert_within(h[some], act64(1, gd) * ud, eg * (ud.abs() + eu) + gd.abs() * eu + 2.0 ** -23 * (gd * ud).abs(), 1)
    dwu, dx = torch.empty_like(wu), torch.empty_like(x)
    ws, n = workspace(z, T, K, N, True, True)
    z.zero_gated_backward(h, N, g, N, u, N, x, K, wg, K, wu, K, dx, K, None, 0, dwu, K, None, None, T, K, N, 1, 1, ws, n)
    du = lambda r: h[r].double() * act64(1, g[r].double())  # noqa: E731
    dg = torch.where(g[some].double() > 0, h[some].double() * u[some].double(), 0.0)
    ref = dg @ wg.double() + du(some) @ wu.double()
    mag = dg.abs() @ wg.double().abs() + du(some).abs() @ wu.double().abs()
    assert_within(dx[some], ref, (2.0 ** -8 + (2 * N + 8) * 2.0 ** -23) * mag, 1)
    cols = torch.arange(0, N, 1000, device="cuda")
    ref = mag = 0
    for r in range(0, T, 30000):
        d = h[r:r + 30000, cols].double() * act64(1, g[r:r + 30000, cols].double())
        ref, mag = ref + d.T @ x[r:r + 30000].double(), mag + d.abs().T @ x[r:r + 30000].double().abs()
    assert_within(dwu[cols], ref, (2.0 ** -8 + (T + 8) * 2.0 ** -23) * mag, 1)
