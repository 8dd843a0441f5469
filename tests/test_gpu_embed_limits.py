"""The embedding's gradient with the longest chunks (from 65536 tokens and columns on), and with vocabularies of four digits.
Tolerances: those of test_gpu_embed.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, NAN, assert_within, rows  # noqa: E402
from test_gpu_embed import check_grad, z  # noqa: E402,F401


@pytest.mark.parametrize("T,D,V,kind", [(800003, 8, 5000, "any"), (1000001, 24, 7, "frequent"), (400001, 520, 900, "frequent"), (700001, 600, 3000, "any"),
                                        (500000, 1100, 2, "same"), (700001, 600, 20, "none")])
@pytest.mark.parametrize("ty,pad,shift,add", [(1, 0, 0, False), (0, 0, 0, True), (1, 3, 1, True), (0, 1, 0, False)])
def test_long_chunks(z, T, D, V, kind, ty, pad, shift, add):  # noqa: F811
    """Chunks of 96, 128 and 256 tokens, whole ones within one run, runs that pass many of them."""
    check_grad(z, T, D, V, kind, ty, pad, shift, add, seed=D)


@pytest.mark.parametrize("V", [(1 << 27) - 1, 1 << 27, (1 << 28) + 5, 1 << 30])
@pytest.mark.parametrize("T", [1, 700, 9000, 70000])
def test_four_digits(z, T, V):  # noqa: F811
    """Three and four passes of the sort, by one cluster and by launches; ids at both ends of every digit."""
    D = 1
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    edges = [0, V - 1, -1, 511, 512, (1 << 18) - 1, 1 << 18, (1 << 27) - 2, V // 2, V // 2 + 1, 2 ** 31 - 1, V - 1, 0]
    ids[:len(edges)] = torch.tensor(edges[:T], device="cuda").int()
    dy, _ = rows(T, D, 0, DT[0], gen)
    dt = torch.full((V, D), NAN, dtype=DT[0], device="cuda")
    n = z.zero_embed_workspace(T, D, V)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    z.zero_embed_backward(ids, dy, D, dt, D, T, D, V, 1.0, False, 0, ws, n)
    there = (ids >= 0) & (ids < V)
    used, where = torch.unique(ids[there].long(), return_inverse=True)
    zero = torch.zeros((len(used), D), dtype=torch.float64, device="cuda")
    ref, mag = (zero.index_add(0, where, f(dy[there].double())) for f in (lambda x: x, torch.abs))
    assert_within(dt[used], ref, (T + 2) * 2.0 ** -24 * mag, 0)
    dt[used] = 0
    assert int(torch.count_nonzero(dt)) == 0 and not bool(torch.isnan(dt[:1000]).any())
