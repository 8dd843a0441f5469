"""Arguments that the AdamW step refuses before any CUDA call (made-up addresses: only where no kernel can run)."""
import ctypes

import pytest

from conftest import cuda_available
from test_train_abi import BASE, plan, rows

no_gpu = pytest.mark.skipif(cuda_available(), reason="made-up addresses: only where no kernel can run")


@no_gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_an_epsilon_below_the_normal_range_is_refused(zlib, bits):
    """Its reciprocal has no fp32 value, and the update of a weight with a zero variance divides by it alone."""
    z = zlib
    rc, info = plan(z, rows(z, 1), bits=bits)
    assert rc == 0
    step = lambda eps: z.lib().zero_adamw_step(ctypes.byref(info), BASE, None, 1, 1e-3, 0.9, 0.999, eps, 0, None)  # noqa: E731
    for eps in (1e-45, 1e-40, 1.1754942e-38):
        assert step(eps) == z.ZERO_EINVAL, eps
    for eps in (0.0, 1.1754944e-38, 1e-8):  # passes the checks, ends at the missing device
        assert step(eps) == z.ZERO_ECUDA, eps
