"""The layers where their memory paths change: every phase of a row and every matrix on a phase of its own, the smallest rows,
the sizes at which another kernel takes over, calls on two streams at once.  Tolerances as in the layers' own tests."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, HALF_ULP, NAN, SUB, assert_within, outside_untouched, rows  # noqa: E402
from test_gpu_embed import check_grad, tokens  # noqa: E402


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    yield zlib
    assert zlib.zero_train_timeouts() == 0


PHASES = [(0, 0, 1, 3), (3, 1, 0, 0), (1, 5, 2, 7), (8, 0, 5, 2), (7, 6, 7, 6)]   # pad and shift of what is read, of what is written


@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 40, 250, 257, 264, 1025])
@pytest.mark.parametrize("pa,sa,pb,sb", PHASES)
def test_embed_phases(z, D, pa, sa, pb, sb):
    T, V = 61, 23
    gen = torch.Generator(device="cuda").manual_seed(D)
    ids = tokens("frequent", T, V, gen)
    ids[:3] = torch.tensor([2 ** 31 - 1, -2 ** 31, V], device="cuda", dtype=torch.int64).int()
    table, _ = rows(V, D, pa, DT[0], gen, 0.5, sa)
    y, buf = rows(T, D, pb, DT[0], gen, 0.0, sb)
    z.zero_embed_forward(ids, table, D + pa, y, D + pb, T, D, V, 1.0, 0)
    there = (ids >= 0) & (ids < V)
    assert torch.equal(y, torch.where(there[:, None], table[ids.long().clamp(0, V - 1)], torch.zeros((), dtype=DT[0], device="cuda")))
    assert outside_untouched(y, buf)
    for add in (False, True):
        dy, _ = rows(T, D, pa, DT[0], gen, 0.5, sa)
        dt, buf = rows(V, D, pb, DT[0], gen, 0.5, sb)
        old = dt.double()
        dy[~there] = NAN
        n = z.zero_embed_workspace(T, D, V)
        ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
        z.zero_embed_backward(ids, dy, D + pa, dt, D + pb, T, D, V, 1.0, add, 0, ws, n)
        torch.cuda.synchronize()
        zero = torch.zeros((V, D), dtype=torch.float64, device="cuda")
        ref, mag = (zero.index_add(0, ids[there].long(), f(dy[there].double())) for f in (lambda x: x, torch.abs))
        err = (T + 2) * 2.0 ** -24 * mag
        if add:
            ref, err = ref + old, err + 2.0 ** -24 * (ref.abs() + old.abs())
        assert_within(dt, ref, err, 0)
        assert outside_untouched(dt, buf)


@pytest.mark.parametrize("T", [8192, 8193, 16385, 32768, 32769, 65536, 65537])
def test_sorts_take_over_from_each_other(z, T):
    check_grad(z, T, 24, 3000, "frequent", 1, seed=T)
    check_grad(z, T, 9, 513, "any", 0, pad=2, add=True, seed=T)


@pytest.mark.parametrize("V", [1, 511, 512, 513, 262143, 262144, 300000])
def test_digits_of_the_vocabulary(z, V):
    """Ids at both ends of every digit, as many passes as V takes."""
    T, D = 700, 16
    gen = torch.Generator(device="cuda").manual_seed(V)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    ids[:4] = torch.tensor([0, V - 1, V, -1], device="cuda").int()
    dy, _ = rows(T, D, 0, DT[0], gen)
    dt = torch.full((V, D), NAN, dtype=DT[0], device="cuda")
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_embed_backward(ids, dy, D, dt, D, T, D, V, 1.0, False, 0, ws, n)
    there = (ids >= 0) & (ids < V)
    zero = torch.zeros((V, D), dtype=torch.float64, device="cuda")
    ref, mag = (zero.index_add(0, ids[there].long(), f(dy[there].double())) for f in (lambda x: x, torch.abs))
    assert_within(dt, ref, (T + 2) * 2.0 ** -24 * mag, 0)


@pytest.mark.parametrize("D", [1, 2, 5, 8, 9, 63, 64, 65, 128, 129, 250, 257, 512, 1000, 1030, 3000])
@pytest.mark.parametrize("pa,sa,pb,sb", PHASES)
def test_layernorm_phases(z, D, pa, sa, pb, sb):
    """x, dy, the residual's gradient and the outputs in rows of their own strides and phases, weights anywhere."""
    T = 37
    gen = torch.Generator(device="cuda").manual_seed(D)
    dt = DT[0]
    x, _ = rows(T, D, pa, dt, gen, 1.0, sa, 0.2)
    dy, _ = rows(T, D, pb, dt, gen, 0.5, sa)
    res, _ = rows(T, D, pa, dt, gen, 0.5, sb)
    w, b = ((torch.randn(D + 8, generator=gen, device="cuda") * 0.2 + k).to(dt)[s:s + D] for k, s in ((1, sb), (0, sa)))
    y, ybuf = rows(T, D, pb, dt, gen, 0.0, sb)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    z.zero_layernorm_forward(x, D + pa, w, b, y, D + pb, mean, rstd, T, D, 1e-3, 0)
    xd, wd = x.double(), w.double()
    m = xd.mean(1, keepdim=True)
    s = (((xd - m) ** 2).mean(1, keepdim=True) + 1e-3) ** -0.5
    c = 128 * 2.0 ** -24
    h = (xd - m) * s
    em = c * xd.abs().mean(1, keepdim=True)
    err = (em * s + h.abs() * (2 * c + em ** 2 * s ** 2 + 2.0 ** -21) + 2.0 ** -22 * (xd.abs() + m.abs()) * s) * wd.abs() + 2.0 ** -22
    assert_within(y, h * wd + b.double(), err, 0)
    assert outside_untouched(y, ybuf)
    dx, buf = rows(T, D, pb, dt, gen, 0.0, sa)
    dw, db = (torch.full((D + 8,), NAN, dtype=dt, device="cuda")[k:k + D] for k in (sa, sb))
    n = z.zero_layernorm_workspace(T, D)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    z.zero_layernorm_backward(dy, D + pb, x, D + pa, w, mean, rstd, res, D + pa, dx, D + pb, dw, db, T, D, 0, ws, n)
    m, s = mean.double()[:, None], rstd.double()[:, None]
    h, H, dyd = (xd - m) * s, (xd.abs() + m.abs()) * s, dy.double()
    a = dyd * wd
    c1 = (a * h).mean(1, keepdim=True)
    ref = s * (a - a.mean(1, keepdim=True) - h * c1) + res.double()
    err = s * (2.0 ** -22 * a.abs() + 2 * c * a.abs().mean(1, keepdim=True) + H * 2.0 ** -22 * c1.abs()
               + h.abs() * (2 * c + 2.0 ** -22) * (a.abs() * H).mean(1, keepdim=True)) + 2.0 ** -21 * (ref.abs() + res.double().abs())
    assert_within(dx, ref, err, 0, "dx")
    assert_within(dw, (dyd * h).sum(0), (T + 64) * 2.0 ** -23 * (dyd.abs() * H).sum(0), 0, "dw")
    assert_within(db, dyd.sum(0), (T + 64) * 2.0 ** -24 * dyd.abs().sum(0), 0, "db")
    assert outside_untouched(dx, buf)


@pytest.mark.parametrize("D", [3, 9, 70, 300, 1001, 2047, 5001])
def test_layernorm_in_place_off_16_bytes(z, D):
    """y over x and dx over dy or the residual's gradient, in rows whose ends share 16 bytes with their neighbours: the same
    bits as into another matrix."""
    T = 400
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, _ = rows(T, D, 0, DT[1], gen, 1.0, 1)
    dy, res = rows(T, D, 0, DT[1], gen, 1.0, 1)[0], rows(T, D, 0, DT[1], gen, 1.0, 1)[0]
    y, dx = rows(T, D, 0, DT[1], gen, 0.0, 1)[0], rows(T, D, 0, DT[1], gen, 0.0, 1)[0]
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    z.zero_layernorm_forward(x, D, None, None, y, D, mean, rstd, T, D, 1e-5, 1)
    z.zero_layernorm_backward(dy, D, x, D, None, mean, rstd, res, D, dx, D, None, None, T, D, 1)
    for over in (dy, res):
        keep = over.clone()
        z.zero_layernorm_backward(dy, D, x, D, None, mean, rstd, res, D, over, D, None, None, T, D, 1)
        assert torch.equal(over, dx)
        over.copy_(keep)
    z.zero_layernorm_forward(x, D, None, None, x, D, mean, rstd, T, D, 1e-5, 1)
    assert torch.equal(x, y)


@pytest.mark.parametrize("T,K,N", [(3, 100, 50), (150, 130, 70), (300, 264, 520), (5000, 72, 520)])
@pytest.mark.parametrize("off", range(11))
def test_gated_operands_on_phases_of_their_own(z, T, K, N, off):
    """One operand or output at a time off 16 bytes, the others on it: the same bits as with all on it (what a copy lays out is
    the same operand) for fp32 sums in the same order."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    dt = DT[1]
    full = [torch.randn((n, k), generator=gen, device="cuda").to(dt) * s for n, k, s in
            ((T, K, 1.0), (N, K, K ** -0.5), (N, K, K ** -0.5), (T, N, 0.5))]
    bias = [torch.randn(N, generator=gen, device="cuda").to(dt) for _ in range(2)]
    got = []
    for which in (-1, off):
        def place(j, t):
            pad = 8 - t.shape[1] % 8 if j != which else 9 - t.shape[1] % 8
            v = torch.as_strided(torch.zeros(t.shape[0] * (t.shape[1] + pad) + 32, dtype=dt, device="cuda"), t.shape, (t.shape[1] + pad, 1), 1 if j == which else 0)
            return v.copy_(t)
        x, wg, wu, dh = (place(j, t) for j, t in enumerate(full))
        h, g, u = (place(4 + j, torch.zeros((T, N), device="cuda")) for j in range(3))
        dx, dwg, dwu = (place(7 + j, torch.zeros(s, device="cuda")) for j, s in enumerate(((T, K), (N, K), (N, K))))
        bg = bias[0] if which != 10 else torch.cat([bias[0][:1], bias[0]])[1:]
        dbg, dbu = torch.empty(N + 1, dtype=dt, device="cuda")[(which == 10):][:N], torch.empty(N, dtype=dt, device="cuda")
        n = z.zero_gated_workspace(T, K, N, True, False)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        ld = lambda t: t.stride(0)  # noqa: E731
        z.zero_gated_forward(x, ld(x), wg, ld(wg), wu, ld(wu), bg, bias[1], h, ld(h), g, ld(g), u, ld(u), T, K, N, 3, 1, ws, n)
        z.zero_gated_backward(dh, ld(dh), g, ld(g), u, ld(u), x, ld(x), wg, ld(wg), wu, ld(wu), dx, ld(dx), dwg, ld(dwg), dwu, ld(dwu), dbg, dbu, T, K, N, 3, 1, ws, n)
        torch.cuda.synchronize()
        got.append([t.clone() for t in (h, g, u, dx, dwg, dwu, dbg, dbu)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_loss_of_rows_on_every_phase(z):
    """An odd stride: each row starts on another phase; logits and gradient on the same and on different ones."""
    T, V, K = 16, 301, 5
    gen = torch.Generator(device="cuda").manual_seed(9)
    base = torch.randn((T, V), generator=gen, device="cuda").to(DT[1])
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    index = torch.randint(0, V, (T, K), generator=gen, device="cuda").int()
    teacher = torch.randn((T, K), generator=gen, device="cuda")
    want = None
    for pa, sa, pb, sb in [(3, 0, 3, 0)] + PHASES:
        s, _ = rows(T, V, pa, DT[1], gen, 0.0, sa)
        s.copy_(base)
        ds, buf = rows(T, V, pb, DT[1], gen, 0.0, sb)
        loss = torch.empty(T, device="cuda")
        z.zero_distill_loss(s, V + pa, targets, index, teacher, K, None, loss, ds, V + pb, T, V, K, 1.5, 0.5, 1.0, 1)
        assert outside_untouched(ds, buf)
        if want is None:
            want = loss.clone(), ds.clone()
        # sums in another order: a few fp32 steps, and a step of bf16 where that crosses a border
        assert bool(((loss - want[0]).abs() <= 2.0 ** -18 * want[0].abs()).all())
        err = 2.0 ** -17 * want[1].double().abs()
        assert bool(((ds.double() - want[1].double()).abs() <= 2 * HALF_ULP[1] * want[1].double().abs() + err + SUB[1]).all())


def test_two_streams_at_once(z):
    """The layers on two streams with workspaces of their own, interleaved: the bits of calls one after the other."""
    T, D, V, N = 3000, 264, 2000, 200
    gen = torch.Generator(device="cuda").manual_seed(4)
    sets, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        ids = tokens("frequent", T, V, gen)
        x, dy = rows(T, D, 0, DT[1], gen)[0], rows(T, D, 0, DT[1], gen)[0]
        w = rows(2 * N, D, 0, DT[1], gen, D ** -0.5)[0]
        out = [torch.zeros((V, D), dtype=DT[1], device="cuda"), torch.zeros((T, D), dtype=DT[1], device="cuda"), torch.zeros(D, dtype=DT[1], device="cuda"),
               torch.zeros((T, N), dtype=DT[1], device="cuda"), torch.zeros((T, 2 * N), dtype=DT[1], device="cuda"), torch.zeros((2 * N, D), dtype=DT[1], device="cuda"),
               torch.zeros((T, D), dtype=DT[1], device="cuda")]
        mean, rstd = x.float().mean(1), 1 / x.float().std(1)
        need = [z.zero_embed_workspace(T, D, V), z.zero_layernorm_workspace(T, D), z.zero_gated_workspace(T, D, N, True, True)]
        sets.append((ids, x, dy, w, mean, rstd, out, [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for n in need]))

    def calls(k, stream):
        ids, x, dy, w, mean, rstd, out, ws = sets[k]
        yield lambda: z.zero_embed_backward(ids, dy, D, out[0], D, T, D, V, 1.0, False, 1, ws[0], ws[0].numel(), stream=stream)
        yield lambda: z.zero_layernorm_backward(dy, D, x, D, None, mean, rstd, None, 0, out[1], D, out[2], None, T, D, 1, ws[1], ws[1].numel(), stream=stream)
        yield lambda: z.zero_gated_forward(x, D, w, D, w[N:], D, None, None, out[3], N, out[4], 2 * N, out[4][:, N:], 2 * N, T, D, N, 2, 1, ws[2], ws[2].numel(), stream=stream)
        yield lambda: z.zero_gated_backward(out[3], N, out[4], 2 * N, out[4][:, N:], 2 * N, x, D, w, D, w[N:], D, out[6], D, out[5], D, out[5][N:], D, None, None, T, D, N, 2, 1,
                                            ws[2], ws[2].numel(), stream=stream)

    for k in range(2):
        for f in calls(k, None):
            f()
    torch.cuda.synchronize()
    want = [[t.clone() for t in s[6]] for s in sets]
    for _ in range(5):
        for s in sets:
            for t in s[6]:
                t.zero_()
        torch.cuda.synchronize()
        for a, b in zip(calls(0, streams[0]), calls(1, streams[1])):
            a()
            b()
        torch.cuda.synchronize()
        for s, ref in zip(sets, want):
            assert all(torch.equal(p, q) for p, q in zip(s[6], ref))
