"""The gated projections' gradients where dh times u leaves fp32's range and the activation's slope brings it back.

Tolerances: the slope far out is off by (|g| 2^-23 + 2^-20) of itself (the logistic function's argument, its exponential and
reciprocal; its second term is many times the first there), and dg by two more roundings; db is dg of one token, rounded once."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _layers import DT, assert_within  # noqa: E402
from test_gpu_gated import slope64, z  # noqa: E402,F401


@pytest.mark.parametrize("act,gate", [(3, (-45.0, -50.0, -60.0, -70.0)), (2, (-4.5, -5.0, -5.5, -6.0))])
@pytest.mark.parametrize("dh,u", [(1e25, 1e20), (-1e19, 1e24), (1e38, -1e5), (3e37, 1e2)])
def test_slope_before_the_product(z, act, gate, dh, u):  # noqa: F811
    N, dt = 72, DT[1]
    g = torch.tensor(gate, device="cuda").repeat(N // 4).to(dt)[None]
    d, up = (torch.full((1, N), v, device="cuda").to(dt) for v in (dh, u))
    x, dwg, dbg = torch.ones((1, 1), dtype=dt, device="cuda"), torch.empty((N, 1), dtype=dt, device="cuda"), torch.empty(N, dtype=dt, device="cuda")
    n = z.zero_gated_workspace(1, 1, N, True, False)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    z.zero_gated_backward(d, N, g, N, up, N, x, 1, None, 0, None, 0, None, 0, dwg, 1, None, 0, dbg, None, 1, 1, N, act, 1, ws, n)
    torch.cuda.synchronize()
    ref = (d.double() * up.double() * slope64(act, g.double()))[0]
    lost = (g.double().abs() ** (3 if act == 2 else 1) * 2.0 ** -23 + 2.0 ** -20)[0] * 2
    keep = ref.abs() < 3e38
    assert bool(keep.any())
    assert_within(dbg[keep], ref[keep], lost[keep] * ref[keep].abs(), 1, "dbg")
    assert_within(dwg[keep, 0], ref[keep], lost[keep] * ref[keep].abs(), 1, "dwg")
