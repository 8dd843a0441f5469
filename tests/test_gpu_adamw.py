"""AdamW over many tensors (moments in 32 and in 8 bits) and the gradient norm,
against the formulas in 64 bits.

Tolerances come from the operations: every fp32 operation is off by at most
u = 2^-24 of its result, so each quantity below is bounded by the number of
roundings on its way times u times the sum of the magnitudes that enter it."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {0: torch.float16, 1: torch.bfloat16, 2: torch.float32}
LR, B1, B2, EPS = 1e-2, 0.9, 0.999, 1e-8


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def f32(x):
    return float(np.float32(x))


class Case:
    """Tensors in arenas with gaps, sentinels in the gaps, and what the step should make of them."""

    def __init__(self, z, sizes, P, gt, pt, bits, shift=0, stride_pad=0, seed=0, gscale=1e-2, congruent=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.z, self.sizes, self.P, self.bits = z, sizes, P, bits
        offs, at = [], 0
        for k, n in enumerate(sizes):
            at = -(-at // 256) * 256 + (0 if bits == 8 and congruent else 256) + shift
            offs.append(at)
            at += n
        total = at + 300
        self.offs, self.total = offs, total
        skew = 0 if congruent else 1
        self.stride = -(-total // 8) * 8 + stride_pad
        self.graw = torch.empty(P * self.stride + 16, dtype=DT[gt], device="cuda")
        self.graw.copy_(torch.randn(self.graw.shape, generator=gen, device="cuda") * gscale)
        self.g = torch.as_strided(self.graw, (P, total), (self.stride, 1), skew)
        self.master = torch.randn(total, generator=gen, device="cuda")
        self.param = torch.full((total,), float("nan"), dtype=DT[pt], device="cuda")
        self.ms = self.vs = None
        if bits == 32:
            self.m = torch.randn(total, generator=gen, device="cuda") * 1e-3
            self.v = torch.rand(total, generator=gen, device="cuda") * 1e-5
        else:
            self.m = torch.randint(0, 256, (total,), generator=gen, device="cuda").to(torch.uint8)
            self.m[(self.m & 0x7F) == 0x7F] = 0x12            # no NaN codes
            self.v = torch.randint(0, 0x7F, (total,), generator=gen, device="cuda").to(torch.uint8)
            nb = total // 256 + 2 * len(sizes) + 4
            self.ms = torch.rand(nb, generator=gen, device="cuda") * 1e-5 + 1e-7
            self.vs = torch.rand(nb, generator=gen, device="cuda") * 1e-5 + 1e-7
        self.so, s = [], 1
        for n in sizes:
            self.so.append(s)
            s += -(-n // 256)
        self.wd = [0.0 if k % 2 else 0.1 for k in range(len(sizes))]
        self.ls = [1.0 if k % 3 else 0.5 for k in range(len(sizes))]
        rows = []
        for k, n in enumerate(sizes):
            o = offs[k]
            rows.append(dict(grad=self.g[0, o:], rank_stride=self.stride, master=self.master[o:], m=self.m[o:], v=self.v[o:],
                             param=self.param[o:], n=n, weight_decay=self.wd[k], lr_scale=self.ls[k]))
            if bits == 8:
                rows[-1].update(m_scale=self.ms[self.so[k]:], v_scale=self.vs[self.so[k]:])
        self.plan = z.zero_adamw_plan(rows, P, gt, pt, bits)

    def state(self):
        return [t.clone() for t in (self.master, self.m, self.v, self.param) + ((self.ms, self.vs) if self.bits == 8 else ())]

    def moments64(self, k, m, v, ms, vs):
        o, n = self.offs[k], self.sizes[k]
        if self.bits == 32:
            return m[o:o + n].double(), v[o:o + n].double()
        b = torch.arange(n, device="cuda") // 256 + self.so[k]
        code = lambda t: t[o:o + n].view(torch.float8_e4m3fn).double()  # noqa: E731
        return code(m) * ms[b].double(), (code(v) * vs[b].double()) ** 2

    def check(self, before, t, factor=1.0):
        w0, m0, v0, p0 = before[:4]
        ms0, vs0 = before[4:] if self.bits == 8 else (None, None)
        b1, b2, lr, eps = f32(B1), f32(B2), f32(LR), f32(EPS)
        r1, c2 = 1 / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
        touched = torch.zeros(self.total, dtype=torch.bool, device="cuda")
        for k, n in enumerate(self.sizes):
            if n == 0:
                continue
            o = self.offs[k]
            touched[o:o + n] = True
            gr = self.g[:, o:o + n].double()
            g, ga = gr.mean(0) * factor, gr.abs().mean(0) * abs(factor)
            m, v = self.moments64(k, m0, v0, ms0, vs0)
            ma = b1 * m.abs() + (1 - b1) * ga                    # magnitudes that enter m
            va = b2 * v + (1 - b2) * ga * ga
            m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
            em, ev = (self.P + 7) * U * ma, (2 * self.P + 12) * U * va
            den = v.sqrt() * c2 + eps
            up = m * r1 / den
            lrj, wd = lr * self.ls[k], self.wd[k]
            w = w0[o:o + n].double() * (1 - lrj * wd) - lrj * up
            # sqrt moves by ev / (2 sqrt v), at most sqrt(ev); the quotient by em / den and up * d(den) / den
            er = torch.minimum(ev / (2 * v.sqrt().clamp(min=1e-300)), ev.sqrt())
            eu = (em * r1 + up.abs() * (er * c2)) / (den - er * c2).clamp(min=eps * 0.5) + 8 * U * up.abs()
            ew = 4 * U * w0[o:o + n].double().abs() + lrj * eu + 4 * U * lrj * up.abs() + 1e-44
            err = (self.master[o:o + n].double() - w).abs()
            assert bool((err <= ew).all()), (k, n, float((err - ew).max()))
            assert torch.equal(self.param[o:o + n], self.master[o:o + n].to(self.param.dtype)), (k, n)
            if self.bits == 32:
                assert bool(((self.m[o:o + n].double() - m).abs() <= em + 1e-44).all()), (k, n)
                assert bool(((self.v[o:o + n].double() - v).abs() <= ev + 1e-44).all()), (k, n)
                continue
            b = torch.arange(n, device="cuda") // 256
            pad = -(-n // 256) * 256 - n
            high = lambda a: torch.nn.functional.pad(a, (0, pad)).view(-1, 256).amax(1)  # noqa: E731
            for x, ex, sc, codes, step in ((m, em, self.ms, self.m, 0.5), (v.sqrt(), er, self.vs, self.v, 1.0)):
                s = sc[self.so[k]:self.so[k] + len(high(m))].double()
                want, slack = high(x.abs()) / 448, high(ex) / 448
                assert bool(((s - want).abs() <= slack + 4 * U * want).all()), (k, n)
                got = codes[o:o + n].view(torch.float8_e4m3fn).double() * s[b]
                # E4M3 neighbours are 2^-3 apart in the relative, 2^-9 of a scale near zero
                grid = torch.maximum(x.abs() / 8, s[b] / 512)
                assert bool(((got - x).abs() <= step * grid * (1 + 1e-4) + ex * 2 + slack[b] * 448).all()), (k, n)
            r = v.sqrt()
            assert bool(((self.v[o:o + n] > 0) | (r < 1e-30)).all())  # a root above 0 never gets the code 0
            assert bool((self.v[o:o + n] < 0x7F).all())
        # nothing between the tensors changes
        for now, was in zip((self.master, self.m, self.v, self.param), before[:4]):
            a, b_ = (x[~touched].view(torch.uint8) for x in (now, was))
            assert torch.equal(a, b_)
        if self.bits == 8:
            last = self.so[-1] + -(-self.sizes[-1] // 256)
            for now, was in ((self.ms, ms0), (self.vs, vs0)):
                assert torch.equal(now[:1], was[:1]) and torch.equal(now[last:], was[last:])


SIZES = [1, 0, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 3]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("P,gt,pt,shift,pad,congruent", [
    (1, 0, 0, 0, 0, True), (1, 1, 1, 0, 0, True), (1, 2, 0, 0, 0, True), (2, 0, 1, 0, 0, True), (3, 1, 0, 0, 0, True),
    (8, 0, 0, 0, 0, True), (5, 2, 1, 0, 0, True), (4, 0, 0, 3, 0, True), (2, 2, 0, 5, 0, True), (3, 0, 0, 0, 3, True),
    (1, 0, 1, 0, 0, False), (2, 2, 1, 1, 1, False), (13, 1, 1, 7, 0, True)])
def test_step(z, bits, P, gt, pt, shift, pad, congruent):
    c = Case(z, SIZES, P, gt, pt, bits, shift, pad, seed=P + 10 * gt, congruent=congruent)
    # the path is the one meant: whole vectors where one phase serves every stream (and blocks of scales start on it)
    want = sum(n > 0 for n in SIZES) if congruent and pad == 0 and (bits == 32 or shift == 0) else 0
    assert c.plan.info.vector_tensors == want
    for t in (1, 2, 500):
        before = c.state()
        z.zero_adamw_step(c.plan, None, t, LR, B1, B2, EPS, t)
        torch.cuda.synchronize()
        c.check(before, t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("P,gt,pt,shift", [(1, 0, 0, 0), (1, 2, 1, 0), (2, 1, 0, 0), (3, 0, 1, 0), (8, 0, 0, 0), (4, 1, 1, 5), (1, 1, 1, 5), (40, 0, 0, 0)])
def test_many_chunks(z, bits, P, gt, pt, shift):
    """Enough chunks for the pipeline of bulk copies (which 32-bit moments take with P = 1; P = 40 has too few stages for
    it), with ragged ends, tiny tensors between, and a skipped step; 32-bit moments also against the vector kernel, tensor
    by tensor, bit for bit."""
    sizes = [4500000, 257, 0, 4300001, 64, 5000, 255]
    c = Case(z, sizes, P, gt, pt, bits, shift, seed=P)
    assert c.plan.info.chunks >= 4096 and c.plan.info.pipeline == (1 if bits == 32 or shift == 0 else 0)
    for t in (1, 20):
        before = c.state()
        z.zero_adamw_step(c.plan, None, t, LR, B1, B2, EPS, t)
        torch.cuda.synchronize()
        c.check(before, t)
    after = c.state()
    if bits == 32:
        for x, y in zip((c.master, c.m, c.v, c.param), before):
            x.copy_(y)
        for k, n in enumerate(sizes):
            o = c.offs[k]
            if n:
                one = z.zero_adamw_plan([dict(grad=c.g[0, o:], rank_stride=c.stride, master=c.master[o:], m=c.m[o:], v=c.v[o:],
                                              param=c.param[o:], n=n, weight_decay=c.wd[k], lr_scale=c.ls[k])], P, gt, pt, bits)
                assert one.info.chunks < 4096
                z.zero_adamw_step(one, None, 20, LR, B1, B2, EPS, 20)
        for x, y in zip(c.state(), after):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    z.zero_adamw_step(c.plan, torch.zeros(3, device="cuda"), 21, LR, B1, B2, EPS, 21)
    for x, y in zip(c.state(), after):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert z.zero_train_timeouts() == 0


def test_paths_agree(z):
    """The same tensors on whole vectors and element by element: the same bits."""
    for bits in (32, 8):
        a = Case(z, [5000, 300], 2, 0, 0, bits, seed=3)
        b = Case(z, [5000, 300], 2, 0, 0, bits, seed=3)
        odd = torch.empty(b.graw.numel() + 1, dtype=torch.float16, device="cuda")[1:]
        odd.copy_(b.graw)                                     # the gradients alone one element off
        rows = []
        for k, n in enumerate(b.sizes):
            o = b.offs[k]
            rows.append(dict(grad=odd[o:], rank_stride=b.stride, master=b.master[o:], m=b.m[o:], v=b.v[o:], param=b.param[o:], n=n,
                             weight_decay=b.wd[k], lr_scale=b.ls[k]))
            if bits == 8:
                rows[-1].update(m_scale=b.ms[b.so[k]:], v_scale=b.vs[b.so[k]:])
        plan = z.zero_adamw_plan(rows, 2, 0, 0, bits)
        assert plan.info.vector_tensors == 0 and a.plan.info.vector_tensors == 2
        z.zero_adamw_step(a.plan, None, 3, LR, B1, B2, EPS, 9)
        z.zero_adamw_step(plan, None, 3, LR, B1, B2, EPS, 9)
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def mix(h):
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


@pytest.mark.parametrize("n,P,gt", [(12000000, 1, 1), (300000, 3, 0), (12000000, 2, 2)])
def test_8_bit_states_bit_for_bit(z, n, P, gt):
    """Codes and scales of two steps against the formulas in separately rounded fp32 torch operations: equal bits, on the
    pipeline and on the vector kernel.  (A code that differed would move the next step's weight by up to a tenth of an
    update.)"""
    c = Case(z, [n], P, gt, 0, 8, seed=n + P)
    o, nb, so, top = c.offs[0], -(-n // 256), c.so[0], torch.tensor(448.0)
    pad = lambda t: torch.nn.functional.pad(t, (0, nb * 256 - n)).view(nb, 256)  # noqa: E731
    one, b1, b2 = np.float32(1), np.float32(B1), np.float32(B2)
    for t in (7, 8):
        m8, v8, ms, vs = c.m[o:o + n].clone(), c.v[o:o + n].clone(), c.ms[so:so + nb].clone(), c.vs[so:so + nb].clone()
        z.zero_adamw_step(c.plan, None, t, LR, B1, B2, EPS, t)
        g = c.g[0, o:o + n].float()
        for r in range(1, P):
            g = g + c.g[r, o:o + n].float()
        if P > 1:
            g = g / torch.full((), P, dtype=torch.float32, device="cuda")
        g = pad(g)
        m = pad(m8.view(torch.float8_e4m3fn).float()) * ms[:, None]
        r = pad(v8.view(torch.float8_e4m3fn).float()) * vs[:, None]
        m = m * float(b1) + g * float(one - b1)
        r = ((r * r) * float(b2) + (g * g) * float(one - b2)).sqrt()
        hm, hr = m.abs().amax(1, keepdim=True), r.amax(1, keepdim=True)
        assert torch.equal(c.ms[so:so + nb], (hm * f32(1 / 448)).view(-1)) and torch.equal(c.vs[so:so + nb], (hr * f32(1 / 448)).view(-1))
        code = (m * (top / hm)).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:n]
        assert torch.equal(c.m[o:o + n], code)
        key = mix((mix(t) + 0x9E3779B9) & 0xFFFFFFFF)
        h = mix((torch.arange(nb * 128, device="cuda") + key) & 0xFFFFFFFF)
        bits = torch.stack((h & 0xFFFF, h >> 16), 1).view(nb, 256).int()
        y = r * (top / hr)
        cut = ((y * 2.0 ** -120).view(torch.int32) + (bits << 4)) >> 20
        code = torch.where(y > 0, cut.clamp(1, 0x7E), 0).to(torch.uint8).view(-1)[:n]
        assert torch.equal(c.v[o:o + n], code)


def test_zero_state_and_zero_gradients(z):
    """The first step from zero moments; elements without a gradient keep their weight (no decay) and zero moments."""
    for bits in (32, 8):
        c = Case(z, [1000, 700], 1, 0, 0, bits, seed=5)
        for s in c.state():
            pass
        c.m.zero_(), c.v.zero_()
        if bits == 8:
            c.ms.zero_(), c.vs.zero_()
        c.graw.zero_()
        w = c.master.clone()
        z.zero_adamw_step(c.plan, None, 1, LR, B1, B2, EPS, 1)
        o, n = c.offs[1], 700                                  # tensor 1 has no decay
        assert torch.equal(c.master[o:o + n], w[o:o + n])
        assert not c.m[o:o + n].any() and not c.v[o:o + n].any()
        if bits == 8:
            assert not c.ms[c.so[1]:c.so[1] + 3].any() and not c.vs[c.so[1]:c.so[1] + 3].any()


def test_stochastic_rounding_has_the_value_as_its_mean(z):
    """Over many seeds the stored root of v averages to the root; the spread of an average of n
    draws between two neighbours at most d apart is at most d / (2 sqrt n)."""
    c = Case(z, [512], 1, 2, 0, 8, seed=6)
    before = c.state()
    n_seeds = 400
    acc = torch.zeros(512, dtype=torch.float64, device="cuda")
    o = c.offs[0]
    for seed in range(n_seeds):
        for t, s in zip((c.master, c.m, c.v, c.param, c.ms, c.vs), before):
            t.copy_(s)
        z.zero_adamw_step(c.plan, None, 100, LR, B1, B2, EPS, seed)
        sc = c.vs[c.so[0]:c.so[0] + 2].double().repeat_interleave(256)
        acc += c.v[o:o + 512].view(torch.float8_e4m3fn).double() * sc
    m, v = c.moments64(0, before[1], before[2], before[4], before[5])
    r = (f32(B2) * v + (1 - f32(B2)) * c.g[0, o:o + 512].double() ** 2).sqrt()
    grid = torch.maximum(r / 8, sc / 512)
    tiny = r < sc / 512                                        # below the first code: always that code
    err = (acc / n_seeds - r).abs()
    assert bool((err[~tiny] <= (5.5 * grid / (2 * math.sqrt(n_seeds)))[~tiny]).all())
    # another tensor index or seed gives other bits, the same gives the same
    for t, s in zip((c.master, c.m, c.v, c.param, c.ms, c.vs), before):
        t.copy_(s)
    z.zero_adamw_step(c.plan, None, 100, LR, B1, B2, EPS, 0)
    first = c.v.clone()
    for t, s in zip((c.master, c.m, c.v, c.param, c.ms, c.vs), before):
        t.copy_(s)
    z.zero_adamw_step(c.plan, None, 100, LR, B1, B2, EPS, 0)
    assert torch.equal(c.v, first)


def test_non_finite_moments_stay_in_their_block(z):
    """A NaN and an infinite gradient: their blocks' states decode to NaN, every other block is as without them."""
    a, b = (Case(z, [1024], 1, 2, 0, 8, seed=8) for _ in range(2))
    o = a.offs[0]
    a.g[0, o + 300] = float("nan")
    a.g[0, o + 600] = float("inf")
    for c in (a, b):
        z.zero_adamw_step(c.plan, None, 2, LR, B1, B2, EPS, 1)
    s = a.so[0]
    assert torch.isnan(a.ms[s + 1:s + 3]).all() and torch.isnan(a.vs[s + 1:s + 3]).all()
    for lo, hi in ((0, 256), (768, 1024)):
        for x, y in zip(a.state()[:4], b.state()[:4]):
            assert torch.equal(x[o + lo:o + hi].view(torch.uint8), y[o + lo:o + hi].view(torch.uint8))


@pytest.mark.parametrize("P,gt,shift,pad", [(1, 0, 0, 0), (1, 1, 3, 0), (1, 2, 1, 1), (4, 0, 0, 0), (3, 1, 0, 3), (8, 2, 0, 0)])
@pytest.mark.parametrize("sizes", [[1], [0], [100000, 7, 0, 8192, 8193], [3000000]])
def test_norm_and_clipping(z, P, gt, shift, pad, sizes):
    c = Case(z, sizes, P, gt, 0, 32, shift, pad, seed=4)
    plan = z.zero_grad_plan([dict(grad=c.g[0, o:], rank_stride=c.stride, n=n) for o, n in zip(c.offs, sizes)], P, gt)
    g = torch.cat([c.g[:, o:o + n].double() for o, n in zip(c.offs, sizes)], 1)
    norm = float((g.mean(0) ** 2).sum().sqrt()) * 0.5
    # each mean is off by (P + 1) u of the magnitudes, its square twice that, the sums of eight and the compensated sum a few u
    slack = float((g.abs().mean(0) ** 2).sum().sqrt()) * 0.5 * (P + 16) * U
    stats = torch.full((3,), -1.0, device="cuda")
    for p in (plan, c.plan):                                   # a step's plan serves the norm too
        for top in (norm / 3 if norm else 1.0, norm * 3 + 1, 0.0):
            z.zero_grad_norm(p, 0.5, top, stats)
            s = stats.cpu().double()
            assert abs(float(s[0]) - norm) <= slack and s[2] == 1.0
            want = 0.5 * min(1.0, top / (norm + 1e-6)) if top > 0 else 0.5
            assert abs(float(s[1]) - want) <= want * ((slack / norm if norm else 0) + 8 * U)
    first = stats.clone()
    z.zero_grad_norm(plan, 0.5, 0.0, stats)
    assert torch.equal(first, stats)                           # the same bits again


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_and_skipped_step(z, bits):
    c = Case(z, SIZES, 2, 0, 0, bits, seed=12)
    stats = torch.zeros(3, device="cuda")
    z.zero_grad_norm(c.plan, 0.25, 0.01, stats)
    before = c.state()
    z.zero_adamw_step(c.plan, stats, 5, LR, B1, B2, EPS, 5)
    factor = float(stats[1])
    assert 0 < factor < 0.25
    c.check(before, 5, factor)
    for bad in (float("inf"), float("nan")):
        c.g[1, c.offs[10] + 4321] = bad
        z.zero_grad_norm(c.plan, 1.0, 1.0, stats)
        assert stats[1] == 0 and stats[2] == 0 and not math.isfinite(float(stats[0]))
        before = c.state()
        z.zero_adamw_step(c.plan, stats, 6, LR, B1, B2, EPS, 6)
        for x, y in zip(c.state(), before):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_other_stream_and_graph(z):
    """A step on a stream of its own, and captured and replayed: the bits of the plain calls."""
    a, b = (Case(z, [5000, 333], 2, 0, 0, 8, seed=2) for _ in range(2))
    sa, sb = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    for t in (1, 1):
        z.zero_grad_norm(a.plan, 1.0, 0.1, sa)
        z.zero_adamw_step(a.plan, sa, t, LR, B1, B2, EPS, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        z.zero_grad_norm(b.plan, 1.0, 0.1, sb, stream=side)
        z.zero_adamw_step(b.plan, sb, 1, LR, B1, B2, EPS, 7, stream=side)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a.state() + [sa], b.state() + [sb]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_large_tensor_offsets(z):
    """More than 2^31 elements in one tensor with 8-bit moments: windows at both ends and across 2^31 against a step
    over copies of them alone (32-bit moments would be the same addressing at four times the size)."""
    n = 2 ** 31 + 4099
    g = torch.empty(n, dtype=torch.float16, device="cuda")
    for lo in range(0, n, 2 ** 28):
        g[lo:lo + 2 ** 28].normal_(0, 1e-2)
    w = torch.ones(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(n // 256 + 1, device="cuda") for _ in range(2))
    p = torch.zeros(n, dtype=torch.float16, device="cuda")
    plan = z.zero_adamw_plan([dict(grad=g, master=w, m=m, v=v, m_scale=ms, v_scale=vs, param=p, n=n, weight_decay=0.1)], 1, 0, 0, 8)
    z.zero_adamw_step(plan, None, 1, LR, B1, B2, EPS, 3)
    for lo in (0, 2 ** 31 - 2048, n // 256 * 256 - 512):
        k = min(4096, n - lo)
        gg = g[lo:lo + k].double()
        mm, r = (1 - f32(B1)) * gg, ((1 - f32(B2)) * gg * gg).sqrt()
        want = 1.0 - f32(LR) * f32(0.1) - f32(LR) * (mm / (1 - f32(B1))) / (r / math.sqrt(1 - f32(B2)) + f32(EPS))
        assert bool(((w[lo:lo + k].double() - want).abs() <= 16 * U).all())
        assert torch.equal(p[lo:lo + k], w[lo:lo + k].half())
        b = (torch.arange(k, device="cuda") + lo) // 256
        assert bool(((m[lo:lo + k].view(torch.float8_e4m3fn).double() * ms[b].double() - mm).abs()
                     <= torch.maximum(mm.abs() / 16, ms[b].double() / 1024) * 1.001).all())


def test_rejected_calls_write_nothing(z):
    c = Case(z, [300], 1, 0, 0, 32, seed=1)
    row = dict(grad=c.g[0], master=c.master, m=c.m, v=c.v, param=c.param, n=300)
    for kw, code in [(dict(n=-1), -1), (dict(master=None), -1), (dict(weight_decay=-0.1), -1), (dict(lr_scale=math.nan), -1),
                     (dict(master=c.master.data_ptr() + 2), -2), (dict(v=c.m), -3), (dict(param=c.graw), -3)]:
        with pytest.raises(z.ZeroError) as e:
            z.zero_adamw_plan([dict(row, **kw)], 1, 0, 0, 32)
        assert e.value.code == code, kw
    before = c.state()
    for args in [(0, LR, B1, B2, EPS), (1, math.inf, B1, B2, EPS), (1, LR, 1.0, B2, EPS), (1, LR, B1, -0.1, EPS), (1, LR, B1, B2, -1.0)]:
        with pytest.raises(z.ZeroError) as e:
            z.zero_adamw_step(c.plan, None, *args)
        assert e.value.code == z.ZERO_EINVAL
    with pytest.raises(z.ZeroError):
        z.zero_adamw_step(z.zero_grad_plan([dict(grad=c.g[0], n=300)], 1, 0), None, 1, LR, B1, B2, EPS)
    stats = torch.full((3,), 7.0, device="cuda")
    for scale, top in ((0.0, 1.0), (math.inf, 1.0), (1.0, math.nan)):
        with pytest.raises(z.ZeroError):
            z.zero_grad_norm(c.plan, scale, top, stats)
    torch.cuda.synchronize()
    assert bool((stats == 7.0).all())
    for x, y in zip(c.state(), before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
