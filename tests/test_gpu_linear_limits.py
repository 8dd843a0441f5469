"""The linear layer at the ends of their ranges: outputs of more than 2^30 columns, infinite and NaN gradients
in places that ReLU masks; matrices on boundaries of their own; the one rounding of dz."""
import math
import random

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


def placed(rows, width, dt, gen, scale, ld, shift):
    """[rows, width] values in rows of ld elements, `shift` elements into their buffer; NaN around them."""
    buf = torch.full((rows * ld + shift + 16,), math.nan, dtype=dt, device="cuda")
    v = torch.as_strided(buf, (rows, width), (ld, 1), shift)
    return v.copy_(torch.randn((rows, width), generator=gen, device="cuda") * scale), buf


def untouched_around(v, buf):
    keep = buf.clone()
    torch.as_strided(keep, v.shape, v.stride(), v.storage_offset()).fill_(math.nan)
    return bool(torch.isnan(keep).all())


SIZES = [(3, 200, 304), (100, 72, 96), (300, 200, 328), (1100, 512, 264), (5000, 136, 1000)]  # few tokens, tiles, pairs
U16 = {0: 2.0 ** -11, 1: 2.0 ** -8}


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("ty", [0, 1])
def test_every_matrix_on_a_boundary_of_its_own(z, T, K, N, ty):
    """x, w, the residual, y and z each on 16, 4 or 2 bytes, apart from the others (in place residuals too).  Tolerances:
    (K + 8) 2^-23 of the sum of magnitudes for the product, one rounding to 16 bits (fp16's subnormals: 2^-25)."""
    rng = random.Random(T + ty)
    dt, u = (torch.float16, torch.bfloat16)[ty], U16[ty]
    gen = torch.Generator(device="cuda").manual_seed(T)
    places = [(0, 0), (0, 0), (8, 8), (2, 0), (0, 2), (1, 0), (0, 1), (3, 5)]  # elements of padding, of shift
    for turn in range(12):
        px, pw, pr, py, pz = (rng.choice(places) for _ in range(5))
        inplace, act = turn % 3 == 2, turn % 4
        x, _ = placed(T, K, dt, gen, 1.0, K + px[0], px[1])
        w, _ = placed(N, K, dt, gen, K ** -0.5, K + pw[0], pw[1])
        b = placed(1, N, dt, gen, 1.0, N, rng.choice([0, 1, 8]))[0][0]
        y, ybuf = placed(T, N, dt, gen, 1.0, N + py[0], py[1])
        r, pr = (y, py) if inplace else (placed(T, N, dt, gen, 1.0, N + pr[0], pr[1])[0], pr)
        rd = r.double()
        pre, zbuf = placed(T, N, dt, gen, 0.0, N + pz[0], pz[1])
        n = z.zero_linear_workspace(T, K, N, act, False, False)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        z.zero_linear_forward(x, K + px[0], w, K + pw[0], b, r, N + pr[0], y, N + py[0], pre, N + pz[0], T, K, N, act, ty, ws, n)
        zd = x.double() @ w.double().T + b.double()
        ez = (K + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T + b.double().abs()) + 2.0 ** -40
        yd = (zd, zd.clamp(min=0), torch.nn.functional.gelu(zd, approximate="tanh"), zd * torch.sigmoid(zd))[act] + rd
        ey = 1.13 * ez + (2.0 ** -18 * (zd.abs() + 1) if act > 1 else 0) + 2.0 ** -23 * yd.abs()
        for got, want, e, buf, name in ((y, yd, ey, ybuf, "y"), (pre, zd, ez, zbuf, "z")):
            bad = (got.double() - want).abs() - (e + u * (want.abs() + e) + (2.0 ** -25 if ty == 0 else 0))
            assert float(bad.max()) <= 0 and untouched_around(got, buf), (name, turn, px, pw, pr, py, pz, inplace, act)


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("ty", [0, 1])
def test_every_gradient_on_a_boundary_of_its_own(z, T, K, N, ty):
    """The same for dy, z, x, w and the outputs dx, dw and db: the bits of the gradients from matrices on 16 bytes."""
    rng = random.Random(T + 7 * ty)
    dt = (torch.float16, torch.bfloat16)[ty]
    gen = torch.Generator(device="cuda").manual_seed(T)
    shapes = dict(dy=(T, N, 0.5), z=(T, N, 1.0), x=(T, K, 1.0), w=(N, K, K ** -0.5), dx=(T, K, 0.0), dw=(N, K, 0.0), db=(1, N, 0.0))
    values = {k: placed(r, c, dt, gen, s, c, 0)[0].clone() for k, (r, c, s) in shapes.items()}
    n = z.zero_linear_workspace(T, K, N, 2, True, False)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def run(place):
        m, bufs = {}, {}
        for k, (r, c, s) in shapes.items():
            m[k], bufs[k] = placed(r, c, dt, gen, 0.0, c + (0 if k == "db" else place[k][0]), place[k][1])
            m[k].copy_(values[k])
        ld = {k: c + place[k][0] for k, (_, c, _) in shapes.items()}
        z.zero_linear_backward(m["dy"], ld["dy"], m["z"], ld["z"], m["x"], ld["x"], m["w"], ld["w"], m["dx"], ld["dx"], m["dw"], ld["dw"],
                               m["db"], T, K, N, 2, ty, ws, n)
        for k in ("dx", "dw", "db"):
            assert untouched_around(m[k], bufs[k]), (k, place)
        return [m[k].clone() for k in ("dx", "dw", "db")]

    want = run({k: (-(-c // 8) * 8 - c, 0) for k, (_, c, _) in shapes.items()})
    for turn in range(12):
        place = {k: rng.choice([(0, 0), (8, 8), (2, 0), (0, 2), (1, 0), (0, 1), (3, 5)]) for k in shapes}
        for a, b in zip(run(place), want):
            assert torch.equal(a, b), place


@pytest.mark.parametrize("act,ty", [(2, 0), (2, 1), (3, 1), (0, 1)])
@pytest.mark.parametrize("T,K,N", [(2048, 512, 1024), (77, 136, 264)])
def test_gradients_are_those_of_dz_rounded_once(z, T, K, N, act, ty):
    """The gradients against the formulas with dz rounded to the type once, as the header has it: the same bits in every
    call, and no further off than the roundings of dz that fall otherwise.  A dz whose fp32 value is off by a few 2^-23
    falls to the other neighbour, twice the largest error away, in less than one case of 192; of N (T) independent ones
    the sums are then off by less than 2 sqrt(3 / 192) = 1/4 of what the roundings themselves do."""
    dt = (torch.float16, torch.bfloat16)[ty]
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, w, dy, pre = ((torch.randn(s, generator=gen, device="cuda") * k).to(dt) for s, k in (((T, K), 1), ((N, K), 0.05), ((T, N), 0.1), ((T, N), 1)))
    n = z.zero_linear_workspace(T, K, N, act, True, True)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    runs = []
    for _ in range(3):
        dx, dw, db = (torch.full(s, math.nan, dtype=dt, device="cuda") for s in ((T, K), (N, K), (N,)))
        z.zero_linear_backward(dy, N, pre if act else None, N, x, K, w, K, dx, K, dw, K, db, T, K, N, act, ty, ws, n)
        runs.append((dx, dw, db))
    for again in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], again))
    p = pre.double().requires_grad_()
    y = (p, None, torch.nn.functional.gelu(p, approximate="tanh"), p * torch.sigmoid(p))[act]
    dz = torch.autograd.grad(y, p, dy.double())[0]
    rounded = dz.to(dt).double()
    rms = lambda a: float(a.square().mean().sqrt())  # noqa: E731
    for got, f in ((runs[0][0], lambda d: d @ w.double()), (runs[0][1], lambda d: d.T @ x.double())):
        want = f(rounded)
        moved = rms(want - f(dz)) if act else 0.0
        # the result's own rounding is spread evenly within half an ulp, at most u of it; fp32's sums are off by far less
        u = (2.0 ** -11, 2.0 ** -8)[ty]
        off = rms(got.double() - want)
        assert off <= rms(want) * (u / math.sqrt(3) + 2.0 ** -18) + moved / 4, (off, moved)
    assert bool((runs[0][2].double() - dz.sum(0)).abs().le((T + 8) * 2.0 ** -18 * dz.abs().sum(0) + (2.0 ** -11, 2.0 ** -8)[ty] * dz.sum(0).abs() + 2.0 ** -25).all())
