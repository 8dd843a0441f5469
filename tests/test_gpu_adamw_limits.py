"""AdamW and the gradient norm at the ends of their ranges: moments whose squares leave fp32's normal range, gradients whose
squares do, the random bits of every tensor of a list.

AdamW's references are the header's formulas in fp32 with every operation rounded by itself (numpy, which keeps
subnormals); codes and scales have to be equal to theirs bit for bit.  The weight's line has fused products and a
quotient within 2 ulp: it is held to 8 roundings of the update and 4 of the weight (u = 2^-24)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2 = 0.9, 0.999
F = np.float32


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    yield zlib
    assert zlib.zero_train_timeouts() == 0


def mix(h):
    """MurmurHash3's 32-bit finaliser (A. Appleby)."""
    h = np.asarray(h, np.uint64)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & np.uint64(0xFFFFFFFF)
    h = ((h ^ (h >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def widen(codes, scale, n):
    """fp32 values of E4M3 codes and their blocks' scales."""
    x = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()
    return x * np.repeat(scale, 256)[:n]


class List8:
    """Tensors with 8-bit moments on the GPU, and the step's formulas on the host."""

    def __init__(self, z, sizes, grads, m=None, v=None, ms=None, vs=None, shift=0):
        self.z, self.sizes = z, sizes
        self.g = [np.ascontiguousarray(g, F) for g in grads]
        rng = np.random.default_rng(sum(sizes))
        self.w = [rng.standard_normal(n).astype(F) for n in sizes]
        nb = [-(-n // 256) for n in sizes]
        zeros = lambda k, dt: [np.zeros(k[j], dt) for j in range(len(k))]  # noqa: E731
        self.m, self.v = m or zeros(sizes, np.uint8), v or zeros(sizes, np.uint8)
        self.ms, self.vs = ms or zeros(nb, F), vs or zeros(nb, F)

        def put(a):  # `shift` elements into a buffer of its own
            t = torch.empty(a.size + shift + 16, dtype=torch.from_numpy(a).dtype, device="cuda")[shift:shift + a.size]
            return t.copy_(torch.from_numpy(a))

        self.dev = [{k: put(a[j]) for k, a in (("grad", self.g), ("master", self.w), ("m", self.m), ("v", self.v), ("m_scale", self.ms),
                                               ("v_scale", self.vs))} for j in range(len(sizes))]
        rows = []
        for d, n in zip(self.dev, sizes):
            d["param"] = torch.empty(n + shift, dtype=torch.float16, device="cuda")[shift:]
            rows.append(dict(d, n=n))
        self.plan = z.zero_adamw_plan(rows, 1, z.TYPE_FP32, z.TYPE_FP16, 8)

    def formulas(self, j, t, lr, eps, seed):
        """(weight, bound of its error, m codes, v codes, m scales, v scales) of tensor j after the step."""
        n, nb = self.sizes[j], -(-self.sizes[j] // 256)
        b1, b2 = F(B1), F(B2)
        g, w = self.g[j], self.w[j]
        with np.errstate(all="ignore"):
            m = b1 * widen(self.m[j], self.ms[j], n) + (F(1) - b1) * g
            r = widen(self.v[j], self.vs[j], n)
            v = b2 * (r * r) + (F(1) - b2) * (g * g)
            root = np.sqrt(v)
            r1 = F(1 / (1 - float(b1) ** t))
            c2 = F(1 / math.sqrt(1 - float(b2) ** t))
            up = m.astype(np.float64) * float(F(lr) * r1) / (root.astype(np.float64) * float(c2) + float(F(eps)))
            want = w.astype(np.float64) - up
            pad = lambda a: np.pad(a, (0, nb * 256 - n)).reshape(nb, 256)  # noqa: E731
            m, root = pad(m), pad(root)
            hm, hr = np.abs(m).max(1, keepdims=True), root.max(1, keepdims=True)
            tiny = F(2.0 ** -96)
            im, ir = (np.where(h < tiny, F(0), F(448) / h) for h in (hm, hr))
            sm, sr = (np.where(h < tiny, F(0), np.where(np.isfinite(h), h * F(1 / 448), F(np.nan))).reshape(-1) for h in (hm, hr))
            mc = torch.from_numpy((m * im).reshape(-1)[:n]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            h = mix(np.arange(nb * 128, dtype=np.uint64) + mix((int(mix(seed)) + 0x9E3779B9 * (j + 1)) & 0xFFFFFFFF) & np.uint64(0xFFFFFFFF))
            rnd = np.stack((h & np.uint64(0xFFFF), h >> np.uint64(16)), 1).reshape(-1).astype(np.uint32)
            y = (root * ir).reshape(-1)
            cut = ((y * F(2.0 ** -120)).view(np.uint32) + (rnd << np.uint32(4))) >> np.uint32(20)
            vc = np.where(y > 0, np.clip(cut, 1, 0x7E), 0).astype(np.uint8)[:n]
        return want, 8 * U * np.abs(up) + 4 * U * np.abs(w), mc, vc, sm.astype(F), sr.astype(F)

    def step_and_check(self, t, lr, eps, seed):
        self.z.zero_adamw_step(self.plan, None, t, lr, B1, B2, eps, seed)
        for j, n in enumerate(self.sizes):
            if n == 0:
                continue
            want, bound, mc, vc, sm, sr = self.formulas(j, t, lr, eps, seed)
            got = {k: x.cpu().numpy() for k, x in self.dev[j].items()}
            for k, ref in (("m_scale", sm), ("v_scale", sr)):
                assert np.array_equal(got[k], ref, equal_nan=True), (j, k, got[k], ref)
            for k, ref, s in (("m", mc, sm), ("v", vc, sr)):       # a block whose scale is NaN may hold any codes
                ok = np.repeat(~np.isnan(s), 256)[:n]
                assert np.array_equal(got[k][ok], ref[ok]), (j, k, int((got[k] != ref)[ok].sum()))
            err = np.abs(got["master"].astype(np.float64) - want)
            assert bool((err <= bound).all()), (j, float((err - bound).max()))
            with np.errstate(over="ignore"):
                half = got["master"].astype(np.float16)
            assert np.array_equal(got["param"].view(np.uint16), half.view(np.uint16))


def magnitudes(sizes, lo, hi, seed):
    """Gradients of either sign whose blocks of 256 have magnitudes spread over 10^lo .. 10^hi."""
    rng = np.random.default_rng(seed)
    out = []
    for n in sizes:
        e = np.repeat(rng.uniform(lo, hi, -(-n // 256)), 256)[:n]
        out.append((10.0 ** e * rng.uniform(0.5, 1.0, n) * rng.choice([-1.0, 1.0], n)).astype(F))
    return out


LISTS = [([10317, 0, 256, 700], 0), ([10317, 0, 256, 700], 1), ([8400000, 301], 0)]  # vectors, elements, the pipeline


@pytest.mark.parametrize("eps", [0.0, 1e-8])
@pytest.mark.parametrize("sizes,shift", LISTS)
def test_root_of_a_variance_below_the_normal_range(z, sizes, shift, eps):
    """First steps from a zero state with gradients of 1e-20.3 to 1e-15: their squares' thousandth is subnormal below
    3.4e-18, and with eps = 0 the update divides by its root alone."""
    List8(z, sizes, magnitudes(sizes, -20.3, -15, 3), shift=shift).step_and_check(1, 1e-2, eps, 5)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [700, 8400000])
def test_infinite_variance_leaves_the_weight(z, bits, n):
    """A finite gradient whose square is infinite, without stats: m / (inf + eps) is 0, so the weight stays; the block's
    8-bit variance gets the scale NaN, its momentum keeps its scale."""
    rng = np.random.default_rng(n)
    g = (rng.standard_normal(n) * 1e-2).astype(F)
    hit = [3, 300, n - 1]
    g[hit] = [2.5e19, -3e20, 1e25]
    if bits == 8:
        c = List8(z, [n], [g])
        c.step_and_check(1, 1e-2, 1e-8, 2)
        d, w0 = c.dev[0], c.w[0]
        assert bool(torch.isnan(d["v_scale"][[0, 1, (n - 1) // 256]]).all()) and bool(torch.isfinite(d["m_scale"]).all())
    else:
        w0 = rng.standard_normal(n).astype(F)
        d = {k: torch.from_numpy(a).cuda() for k, a in (("grad", g), ("master", w0.copy()), ("m", np.zeros(n, F)), ("v", np.zeros(n, F)))}
        d["param"] = torch.empty(n, dtype=torch.float16, device="cuda")
        z.zero_adamw_step(z.zero_adamw_plan([dict(d, n=n)], 1, z.TYPE_FP32, z.TYPE_FP16, 32), None, 1, 1e-2, B1, B2, 1e-8, 2)
        assert bool(torch.isinf(d["v"][hit]).all())
    w = d["master"].cpu().numpy()
    assert np.isfinite(w).all() and np.array_equal(w[hit], w0[hit])


@pytest.mark.parametrize("sizes,shift", LISTS)
def test_codes_of_a_momentum_at_the_far_end(z, sizes, shift):
    """Blocks whose largest momentum lies between 2^120 and fp32's end: the nearest codes of m * (448 / a)."""
    rng = np.random.default_rng(11)
    m = [rng.integers(0, 0x7F, n).astype(np.uint8) | (rng.integers(0, 2, n).astype(np.uint8) << 7) for n in sizes]
    ms = [(10.0 ** rng.uniform(33.5, 35.85, -(-n // 256))).astype(F) for n in sizes]  # times at most 448
    c = List8(z, sizes, [np.zeros(n, F) for n in sizes], m=m, ms=ms, v=[np.full(n, 0x38, np.uint8) for n in sizes],
              vs=[np.full(-(-n // 256), 1.0, F) for n in sizes], shift=shift)
    assert max(float(np.abs(widen(a, s, n)).max()) for a, s, n in zip(m, ms, sizes) if n) > 2.0 ** 127
    c.step_and_check(1000, 1e-30, 1e-8, 7)


NORMS = [(0, 3e4), (0, 6e-8), (1, 1e18), (1, 1.5e19), (1, 1e30), (1, 1e-25), (1, 1e-38), (2, 2e18), (2, 1e37), (2, 3e-24), (2, 1e-41)]


@pytest.mark.parametrize("gt,size", NORMS)
@pytest.mark.parametrize("sizes,P", [([5], 1), ([3000, 7], 3), ([400001, 0, 8192], 1), ([5000000], 2)])
def test_norm_over_the_range_of_its_gradients(z, gt, size, sizes, P):
    """Finite gradients whose squares, or sums of squares, leave fp32's range: the norm is theirs all the same, and the step
    that reads the statistics is not skipped.  Off by (P + 1) u a mean (at least half of the smallest subnormal), twice
    that for its square, the sums of eight and the joins a few u."""
    dt = (torch.float16, torch.bfloat16, torch.float32)[gt]
    gen = torch.Generator(device="cuda").manual_seed(P)
    total = sum(sizes)
    g = ((torch.rand((P, total + 3), generator=gen, device="cuda") + 0.5) * size).to(dt)
    if size > 1:
        g[:, ::7] = 1e-3                                       # small ones among them
    else:
        g[:, ::5] = 0
    if total > 5:                                              # the last quarter's scale is its own
        g[:, total - total // 4:] = g[:, total - total // 4:] * (2.0 ** -30 if size > 1 else 1.0)
    rows, at = [], 0
    for n in sizes:
        rows.append(dict(grad=g[0, at:], rank_stride=total + 3, n=n))
        at += n
    stats = torch.zeros(3, device="cuda")
    z.zero_grad_norm(z.zero_grad_plan(rows, P, gt), 1.0, 1.0, stats)
    mean = g[:, :total].double().mean(0)
    top = float(mean.abs().max())
    norm = float((mean / top).square().sum().sqrt() * top)
    s = stats.double().cpu()
    if norm > torch.finfo(torch.float32).max:                  # the norm itself has no fp32 value
        assert math.isinf(float(s[0])) and float(s[1]) == 0 and float(s[2]) == 0
        return
    assert float(s[2]) == 1.0
    half = 2.0 ** -150 * math.sqrt(total) if P > 1 else 0.0
    assert abs(float(s[0]) - norm) <= norm * (P + 16) * U + half + 2.0 ** -150, (float(s[0]), norm)
    want = min(1.0, 1.0 / (norm + 1e-6))
    assert abs(float(s[1]) - want) <= want * (P + 24) * U + 2.0 ** -149


def test_norm_that_is_not_finite(z):
    """The norm itself above fp32's range, an infinite and a NaN gradient: not finite, factor 0."""
    for fill, bad in ((3e38, 3e38), (1.0, math.inf), (1e30, math.nan), (0.0, -math.inf)):
        g = torch.full((20000,), fill, device="cuda")
        g[12345] = bad
        stats = torch.zeros(3, device="cuda")
        z.zero_grad_norm(z.zero_grad_plan([dict(grad=g, n=20000)], 1, z.TYPE_FP32), 1.0, 1.0, stats)
        s = stats.cpu()
        assert not math.isfinite(float(s[0])) and float(s[1]) == 0 and float(s[2]) == 0


@pytest.mark.parametrize("sizes,shift", [([513, 0, 1, 10317, 0, 256, 700], 0), ([513, 0, 1, 10317, 0, 256, 700], 1), ([0, 4300001, 257, 4200000], 0)])
def test_random_bits_of_every_tensor_and_seed(z, sizes, shift):
    """Codes of several steps over lists with empty tensors and ragged ends, bit for bit: the random bits are those of the
    seed, the tensor's place in the list (empty ones count) and the element.  Tensors of equal states and gradients get
    different codes, and so does another seed."""
    rng = np.random.default_rng(1)
    g = [(rng.standard_normal(n) * 1e-2).astype(F) for n in sizes]
    for seed in (0, 1, 2 ** 32 - 1):
        c = List8(z, sizes, g, shift=shift)
        assert shift or c.plan.info.vector_tensors == sum(n > 0 for n in sizes)
        c.step_and_check(1, 1e-2, 1e-8, seed)
    same = (rng.standard_normal(5000) * 1e-2).astype(F)
    codes = []
    for seed in (4, 4, 5):
        c = List8(z, [5000, 5000], [same, same])
        c.step_and_check(1, 1e-2, 1e-8, seed)
        codes.append([d["v"].cpu().numpy() for d in c.dev])
    assert np.array_equal(codes[0][0], codes[1][0]) and np.array_equal(codes[0][1], codes[1][1])
    # a root lies strictly between two codes almost always, so that other bits round about half of the codes otherwise
    assert (codes[0][0] != codes[0][1]).sum() > 1000 and (codes[0][0] != codes[2][0]).sum() > 1000
