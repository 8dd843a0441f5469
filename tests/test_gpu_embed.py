"""The embedding lookup and its table's gradient against the formulas in 64 bits.

Tolerances.  The lookup is one product in fp32 (2^-24 of itself) and one rounding to 16 bits.  A row of the gradient is a
sum of n rows of dy in fp32, in any order off by at most n 2^-24 times the sum of their magnitudes, times the scale
(2^-24), plus what the table held (2^-24), rounded once."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, NAN, assert_within, outside_untouched, replayed, rows  # noqa: E402


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def tokens(kind, T, V, gen):
    if kind == "same":
        return torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
    if kind == "none":
        return torch.randint(0, 2, (T,), generator=gen, device="cuda").int() * (V + 1) - 1      # -1 and V
    if kind == "distinct":
        return torch.randperm(V, generator=gen, device="cuda")[:T].int()
    if kind == "frequent":                                                                  # few ids often, some not there
        ids = (torch.rand(T, generator=gen, device="cuda").pow(4) * V).int()
        ids[torch.rand(T, generator=gen, device="cuda") < 0.05] = -7
        return ids
    return torch.randint(0, V, (T,), generator=gen, device="cuda").int()


@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (1, 2048, 100), (4, 8, 3), (7, 331, 1000), (300, 1023, 50), (33, 1032, 40), (1000, 64, 70000), (5, 5000, 17)])
@pytest.mark.parametrize("ty,pad,shift,scale", [(0, 0, 0, 1.0), (1, 8, 0, 1.5), (1, 0, 8, -0.3), (0, 3, 1, 45.25)])
def test_lookup(z, T, D, V, ty, pad, shift, scale):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    ids = tokens("frequent", T, V, gen)
    table, _ = rows(V, D, pad, DT[ty], gen, 0.5, shift)
    y, buf = rows(T, D, pad, DT[ty], gen, 0.0, shift)
    z.zero_embed_forward(ids, table, D + pad, y, D + pad, T, D, V, scale, ty)
    there = (ids >= 0) & (ids < V)
    ref = torch.where(there[:, None], table[ids.long().clamp(0, V - 1)].double() * torch.tensor(scale, dtype=torch.float32).double(), 0.0)
    assert_within(y, ref, 2.0 ** -24 * ref.abs(), ty)
    assert outside_untouched(y, buf)


def check_grad(z, T, D, V, kind, ty, pad=0, shift=0, add=False, scale=1.0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = tokens(kind, T, V, gen)
    dy, _ = rows(T, D, pad, DT[ty], gen, 0.5, shift)
    dt, buf = rows(V, D, pad, DT[ty], gen, 0.5, shift)
    old = dt.double()
    there = (ids >= 0) & (ids < V)
    dy[~there] = NAN                                       # what padding holds does not matter
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    z.zero_embed_backward(ids, dy, D + pad, dt, D + pad, T, D, V, scale, add, ty, ws, n)
    torch.cuda.synchronize()
    keep = ids[there].long()
    s = float(torch.tensor(scale, dtype=torch.float32))
    ref = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, keep, dy[there].double()) * s
    mag = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, keep, dy[there].double().abs()) * abs(s)
    count = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, keep, torch.ones(len(keep), dtype=torch.float64, device="cuda"))
    err = (count[:, None] + 2) * 2.0 ** -24 * mag
    if add:
        assert torch.equal(dt[count == 0].double(), old[count == 0])
        ref, err = ref + old, err + 2.0 ** -24 * (ref.abs() + old.abs())
    else:
        assert not bool(dt[count == 0].any())
    assert_within(dt, ref, err, ty)
    assert outside_untouched(dt, buf)


@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (1, 64, 1000), (31, 100, 40), (32, 256, 7), (33, 257, 900), (1024, 331, 513), (1025, 72, 1), (5000, 40, 511), (3000, 264, 300000)])
@pytest.mark.parametrize("kind", ["any", "frequent", "same", "none"])
@pytest.mark.parametrize("ty,pad,shift,add,scale", [(0, 0, 0, False, 1.0), (1, 8, 0, True, 1.5), (0, 3, 1, True, 0.7), (1, 0, 8, False, -2.0)])
def test_gradient(z, T, D, V, kind, ty, pad, shift, add, scale):
    check_grad(z, T, D, V, kind, ty, pad, shift, add, scale, seed=T + D)


@pytest.mark.parametrize("T,D,V,kind", [(20000, 512, 44629, "frequent"), (66000, 64, 5000, "any"), (70001, 40, 2, "any"), (600001, 64, 1000, "frequent"),
                                        (600000, 8, 3, "same"), (8192, 2048, 8192, "distinct"), (150000, 72, 262144, "any")])
@pytest.mark.parametrize("ty,add", [(1, False), (0, True)])
def test_gradient_many_tokens(z, T, D, V, kind, ty, add):
    """Larger sorting blocks, more digits, longer chunks, runs over many chunks."""
    check_grad(z, T, D, V, kind, ty, add=add, seed=V)


def test_no_tokens(z):
    dt = torch.full((10, 24), NAN, dtype=torch.float16, device="cuda")
    z.zero_embed_backward(None, None, 0, dt, 24, 0, 16, 10, 1.0, True, 0)
    assert bool(torch.isnan(dt).all())
    z.zero_embed_backward(None, None, 0, dt, 24, 0, 16, 10, 1.0, False, 0)
    torch.cuda.synchronize()
    assert not dt[:, :16].any() and bool(torch.isnan(dt[:, 16:]).all())
    z.zero_embed_forward(None, None, 16, None, 16, 0, 16, 10, 1.0, 0)


def test_non_finite_rows_stay_in_their_ids(z):
    T, D, V = 500, 72, 40
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = tokens("any", T, V, gen)
    dy, _ = rows(T, D, 0, DT[1], gen)
    a, b = (torch.empty((V, D), dtype=DT[1], device="cuda") for _ in range(2))
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_embed_backward(ids, dy, D, a, D, T, D, V, 1.0, False, 1, ws, n)
    dy[3], dy[4] = NAN, float("inf")
    z.zero_embed_backward(ids, dy, D, b, D, T, D, V, 1.0, False, 1, ws, n)
    ok = torch.ones(V, dtype=torch.bool, device="cuda")
    ok[ids[3].long()] = ok[ids[4].long()] = False
    assert torch.equal(a[ok], b[ok]) and not bool(torch.isfinite(b[ids[3].long()]).any()) and not bool(torch.isfinite(b[ids[4].long()]).any())


def test_graph_repeats_the_bits(z):
    T, D, V = 3001, 264, 1000
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = tokens("frequent", T, V, gen)
    dy, _ = rows(T, D, 0, DT[1], gen)
    dt, y = torch.empty((V, D), dtype=DT[1], device="cuda"), torch.empty((T, D), dtype=DT[1], device="cuda")
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(stream=None):
        z.zero_embed_backward(ids, dy, D, dt, D, T, D, V, 1.0, False, 1, ws, n, stream=stream)
        z.zero_embed_forward(ids, dt, D, y, D, T, D, V, 1.0, 1, stream=stream)

    call()
    torch.cuda.synchronize()
    first = dt.clone(), y.clone()
    again = replayed(call, (dt, y))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_large_offsets(z):
    """A table, its gradient and an output of more than 2^31 elements."""
    V, D, T = 270000, 8192, 600
    table = torch.zeros((V, D), dtype=DT[1], device="cuda")
    ids = torch.cat([torch.arange(V - 300, V), torch.arange(262000, 262300)]).int().cuda()
    table[ids.long()] = torch.randn((T, D), device="cuda").to(DT[1])
    y = torch.empty((T, D), dtype=DT[1], device="cuda")
    z.zero_embed_forward(ids, table, D, y, D, T, D, V, 1.0, 1)
    assert torch.equal(y, table[ids.long()])
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    table.fill_(3.0)
    z.zero_embed_backward(ids, y, D, table, D, T, D, V, 1.0, False, 1, ws, n)
    assert torch.equal(table[ids.long()], y)
    table[ids.long()] = 0
    assert not bool(table[:100].any()) and not bool(table[-1000:].any()) and not bool(table[262140:262150].any())
