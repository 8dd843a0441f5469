"""The loss against targets and a teacher's top logits, and its gradient, against the formulas in 64 bits.

Tolerances.  An exponential 2^(l d) with d = s - (the row's largest) is off by 2^-22 (the hardware's approximation) and
|l d| 2^-23 (its argument, rounded twice), of itself; below 2^-126 it is 0.  A thread adds at most V / 512 + 16 of them
before the threads' sums are joined (at most 30 steps with factors of their own).  So with e = 2^-18 + V 2^-32 every
probability is off by (e + |l d| 2^-22) of itself, log sums by e, and the teacher's by 2^-20; the sums over K add (K + 8) 2^-24."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, NAN, assert_within, outside_untouched, replayed, rows  # noqa: E402

INF = float("inf")


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def plain64(s, targets, index, teacher, weights, tau, alpha, scale):
    """Loss, gradient, and the bounds of their errors before the rounding; one row after the other."""
    T, V = s.shape
    loss, grad = torch.zeros(T, dtype=torch.float64), torch.zeros((T, V), dtype=torch.float64)
    eloss, egrad = torch.zeros_like(loss), torch.zeros_like(grad)
    e = 2.0 ** -18 + V * 2.0 ** -32
    for t in range(T):
        w = float(weights[t]) if weights is not None else 1.0
        if w == 0:
            continue
        x = s[t] - s[t].max()
        far = torch.where(torch.isinf(x), torch.zeros_like(x), x.abs()) * 1.4427
        if alpha < 1 and 0 <= int(targets[t]) < V:
            g = int(targets[t])
            lse = torch.logsumexp(x, 0)
            loss[t] += (1 - alpha) * (lse - x[g])
            eloss[t] += (1 - alpha) * (e + 2.0 ** -22 * (float(lse.abs()) + min(float(far[g]), 1e30)))
            q = torch.exp(x - lse)
            egrad[t] += (1 - alpha) * q * (e + far * 2.0 ** -22)
            q[g] -= 1
            egrad[t, g] += (1 - alpha) * 2.0 ** -22
            grad[t] += (1 - alpha) * q
        if alpha > 0 and index is not None:
            ok = (index[t] >= 0) & (index[t] < V) & (teacher[t] != -INF)
            if bool(ok.any()):
                j, r = index[t][ok].long(), teacher[t][ok].double() / tau
                logp = torch.log_softmax(r, 0)
                lse = torch.logsumexp(x / tau, 0)
                p, logq = logp.exp(), x / tau - lse
                loss[t] += alpha * tau * tau * (p * (logp - logq[j])).sum()
                K = len(j)
                near = torch.where(torch.isinf(logq[j]), torch.zeros_like(logq[j]), logq[j].abs())
                eloss[t] += alpha * tau * tau * (e + (p * (logp.abs() + 1 + near)).sum() * (2.0 ** -19 + K * 2.0 ** -23))
                q = logq.exp()
                egrad[t] += alpha * tau * q * (e + far / tau * 2.0 ** -22)
                q.index_add_(0, j, -p)
                egrad[t].index_add_(0, j, alpha * tau * p * (2.0 ** -19 + (r - r.max()).abs() * 2.0 ** -22 + K * 2.0 ** -23))
                grad[t] += alpha * tau * q
        loss[t] *= w
        eloss[t] *= abs(w)
        grad[t] *= w * scale
        egrad[t] = egrad[t] * abs(w * scale) + 2.0 ** -22 * grad[t].abs() + 1e-37
    return loss, grad, eloss, egrad


def check(z, T, V, K, ty, tau=1.0, alpha=0.5, teacher_type=2, pad=0, shift=0, gpad=None, inplace=False, grad=True, weights=True, masked=0, scale=4.0, twice=False,
          edit=None):
    gen = torch.Generator(device="cuda").manual_seed(T + V + K)
    dt = DT[ty]
    s, sbuf = rows(T, V, pad, dt, gen, 2.5, shift)
    if masked:
        s[:, V - masked:] = -INF
    gpad = pad if gpad is None else gpad
    ds, dbuf = (s, sbuf) if inplace else rows(T, V, gpad, dt, gen, 0.0, shift)
    targets = torch.randint(0, V - masked, (T,), generator=gen, device="cuda").int()
    targets[::5] = -1
    index = teacher = None
    if K:
        index = torch.randint(0, V - masked, (T, K + 3), generator=gen, device="cuda").int()[:, :K]
        if twice and K > 1:
            index[:, 1] = index[:, 0]
            targets[::3] = index[::3, 0]
        teacher = (torch.randn((T, K + 3), generator=gen, device="cuda") * 2).to(DT[teacher_type])[:, :K]
        index[::4, K // 2] = V
        teacher[1::4, 0] = -INF
    wt = torch.rand(T, generator=gen, device="cuda") + 0.5 if weights else None
    if weights:
        wt[::7] = 0
    if edit:
        edit(s, targets, index, teacher, wt)
    loss = torch.full((T + 1,), NAN, device="cuda")
    want = plain64(s.double().cpu(), targets.cpu(), None if index is None else index.cpu(), None if teacher is None else teacher.cpu(), None if wt is None else wt.cpu(),
                   tau, alpha, scale)
    z.zero_distill_loss(s, V + pad, targets, index, teacher, K + 3, wt, loss, ds if grad else None, V + gpad, T, V, K, tau, alpha, scale, ty, teacher_type)
    torch.cuda.synchronize()
    got = loss[:T].double().cpu()
    fine = torch.isfinite(want[0])
    assert torch.equal(got[~fine & ~torch.isnan(want[0])], want[0][~fine & ~torch.isnan(want[0])]) and torch.equal(torch.isnan(got), torch.isnan(want[0]))
    assert bool(((got - want[0]).abs() <= want[2] + 2.0 ** -22 * want[0].abs())[fine].all()), float(((got - want[0]).abs() - want[2])[fine].max())
    assert bool(torch.isnan(loss[T]))
    if grad:
        ref = want[1]
        assert torch.equal(torch.isnan(ds).cpu(), torch.isnan(ref))
        clean = ~torch.isnan(ref).any(1)
        assert_within(ds[clean.cuda()].cpu(), ref[clean], want[3][clean], ty)
        assert outside_untouched(ds, dbuf)


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (1, 2, 2), (5, 7, 3), (9, 100, 20), (11, 1000, 0), (8, 4099, 64), (6, 8192, 513), (5, 10007, 1024), (3, 50001, 8), (2, 150000, 100)])
@pytest.mark.parametrize("ty,tau,alpha,pad,shift", [(0, 1.0, 0.5, 0, 0), (1, 2.0, 0.3, 8, 0), (1, 4.0, 1.0, 1, 0), (0, 1.5, 0.9, 0, 3), (1, 1.0, 0.0, 3, 1)])
def test_loss_and_gradient(z, T, V, K, ty, tau, alpha, pad, shift):
    check(z, T, V, K, ty, tau, alpha, [2, 0, 1][(T + V) % 3], pad, shift)


@pytest.mark.parametrize("kw", [dict(inplace=True), dict(inplace=True, pad=1), dict(grad=False), dict(weights=False), dict(masked=300), dict(masked=993, K=5), dict(gpad=5),
                                dict(twice=True), dict(twice=True, tau=2.0), dict(scale=-1e-3), dict(V=997, inplace=True, shift=1)])
@pytest.mark.parametrize("ty", [0, 1])
def test_forms(z, kw, ty):
    check(z, **{**dict(T=13, V=1000, K=16, ty=ty, tau=1.5, alpha=0.5), **kw})


def test_one_teacher_entry_is_cross_entropy(z):
    """A teacher of one entry, alone: the loss of that entry as the target."""
    T, V = 20, 777
    gen = torch.Generator(device="cuda").manual_seed(0)
    s, _ = rows(T, V, 0, DT[1], gen, 2.0)
    target = torch.randint(0, V, (T, 1), generator=gen, device="cuda").int()
    out = []
    for alpha, K in ((0.0, 0), (1.0, 1)):
        loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
        z.zero_distill_loss(s, V, target, target, torch.zeros((T, 1), device="cuda"), 1, None, loss, ds, V, T, V, K, 1.0, alpha, 1.0, 1)
        out.append((loss, ds))
    assert bool(((out[0][0] - out[1][0]).abs() <= 2.0 ** -20 * out[0][0].abs()).all())
    assert bool(((out[0][1].float() - out[1][1].float()).abs() <= 2.0 ** -7 * out[0][1].float().abs()).all())


def test_rows_without_terms(z):
    """No target, no teacher with a probability, weight 0: loss 0, gradient 0, whatever the logits hold."""
    def edit(s, targets, index, teacher, wt):
        targets[:8] = torch.tensor([-1, 500, 1 << 30, -2 ** 31, 3, -1, -1, 7], device="cuda").int()
        index[:3], teacher[3], index[4], teacher[5] = -1, -INF, 500, -INF
        wt[:8] = torch.tensor([1, 1, 1, 1, 0, 2, 1, 0.0], device="cuda")
        s[0], s[1], s[4], s[7] = NAN, INF, NAN, INF
    for alpha in (0.5, 1.0, 0.0):
        check(z, 12, 500, 10, 1, 2.0, alpha, edit=edit)


def test_infinite_and_nan_logits(z):
    """Masked logits have probability 0; a target or a teacher's token that is masked has an infinite loss; a row that is
    masked altogether, or holds an infinity or NaN, is NaN, and no other row is."""
    def edit(s, targets, index, teacher, wt):
        s[1, 10:] = -INF
        targets[1], index[1] = 3, torch.arange(10, device="cuda").int() % 10
        s[2, 40], targets[2] = -INF, 40
        s[3] = -INF
        s[4, 17] = NAN
        s[5, 18] = INF
        s[6, 5] = -INF
        index[6], teacher[6, 0] = torch.arange(5, 15, device="cuda").int(), 1.0
        teacher[8, 2] = NAN
        index[8] = torch.arange(10, device="cuda").int()
        wt[:10] = 1
        targets[3:9] = 11
    check(z, 12, 600, 10, 1, 2.0, 0.5, edit=edit)
    check(z, 12, 600, 10, 1, 1.0, 0.5, edit=edit)


def test_extreme_logits(z):
    """Logits and teachers as far apart as their types go: no exponential overflows."""
    def edit(s, targets, index, teacher, wt):
        big = torch.finfo(s.dtype).max
        s[1, 0], s[1, 1] = big, -big
        s[2] = big
        s[3] = -big
        teacher[1, 1], teacher[2, 3] = 1e30, -1e30
        targets[1:4] = torch.tensor([0, 5, 9], device="cuda").int()
        index[:, 4:] = torch.arange(20, 26, device="cuda").int()
        index[1], wt[:6] = torch.tensor([0, 2, 3, 4, 5, 6, 7, 8, 9, 10], device="cuda").int(), 1
        teacher[1] = torch.tensor([1e30] + [0.0] * 9, device="cuda")
    check(z, 8, 300, 10, 1, 1.0, 0.5, edit=edit)
    check(z, 8, 300, 10, 0, 2.0, 0.5, edit=edit)


def test_gradient_against_differences(z):
    """Central differences of the summed loss in 64 bits: step h is off by h^2/6 times the third derivative (below 1)."""
    T, V, K, h = 2, 30, 4, 1e-4
    gen = torch.Generator(device="cuda").manual_seed(3)
    s, _ = rows(T, V, 0, DT[0], gen)
    targets = torch.tensor([3, 29], device="cuda").int()
    index = torch.tensor([[3, 5, 7, 9], [1, 1, 2, 8]], device="cuda").int()
    teacher = torch.randn((T, K), generator=gen, device="cuda")
    loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
    z.zero_distill_loss(s, V, targets, index, teacher, K, None, loss, ds, V, T, V, K, 2.0, 0.4, 1.0, 0)
    x = s.double().cpu()
    args = (targets.cpu(), index.cpu(), teacher.cpu(), None, 2.0, 0.4, 1.0)
    for t in range(T):
        for j in range(0, V, 2 if t else 1):
            keep = float(x[t, j])
            x[t, j] = keep + h
            up = plain64(x, *args)[0].sum()
            x[t, j] = keep - h
            down = plain64(x, *args)[0].sum()
            x[t, j] = keep
            got = float(ds[t, j])
            assert abs(got - float(up - down) / (2 * h)) <= 2.0 ** -11 * abs(got) + 2.0 ** -16 + h * h, (t, j)


def test_graph_repeats_the_bits(z):
    T, V, K = 300, 5003, 20
    gen = torch.Generator(device="cuda").manual_seed(2)
    s, _ = rows(T, V, 0, DT[1], gen)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    index = torch.randint(0, V, (T, K), generator=gen, device="cuda").int()
    teacher = torch.randn((T, K), generator=gen, device="cuda")
    loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
    call = lambda stream=None: z.zero_distill_loss(s, V, targets, index, teacher, K, None, loss, ds, V, T, V, K, 2.0, 0.5, 1.0, 1, stream=stream)  # noqa: E731
    call()
    torch.cuda.synchronize()
    first = loss.clone(), ds.clone()
    again = replayed(call, (loss, ds))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_large_offsets(z):
    """Logits of more than 2^31 elements, in place: the last rows."""
    T, V = 33000, 66000
    s = torch.zeros((T, V), dtype=DT[1], device="cuda")
    targets = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    s[-3:] = torch.randn((3, V), generator=gen, device="cuda").to(DT[1])
    targets[-3:] = torch.tensor([0, 500, V - 1], device="cuda").int()
    want = plain64(s[-3:].double().cpu(), targets[-3:].cpu(), None, None, None, 1.0, 0.0, 1.0)
    loss = torch.empty(T, device="cuda")
    z.zero_distill_loss(s, V, targets, None, None, 0, None, loss, s, V, T, V, 0, 1.0, 0.0, 1.0, 1)
    assert bool(((loss[-3:].double().cpu() - want[0]).abs() <= want[2] + 2.0 ** -22 * want[0]).all()) and not bool(loss[:-3].any())
    assert_within(s[-3:].cpu(), want[1], want[3], 1)
    assert not bool(s[:-3:1000].any())
