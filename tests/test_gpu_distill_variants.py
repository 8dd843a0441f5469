"""The loss's kernels by temperature, length of rows and type: which one a call takes is a rule on these, so each of them
is reached here, on both sides of every bound.

Tolerances: those of test_gpu_distill.py, e = 2^-18 + V 2^-32 for a sum, which is (64 + V / 256) 2^-24.  What they have to cover
follows from how many exponentials a thread adds: it has two sums of each kind, so with a teacher V / 64 in a sum below 2560
logits (32 threads go over the row), V / 192 below 16384 (96) and V / 448 above (224), without one V / 128 below 6144 (64
threads), V / 256 below 16384 (128) and V / 512 above (256).  Each addition is off by 2^-24 of the sum so far; the threads' sums
are joined in 12 more; an exponential itself by 2^-22.  A + 12 + 4 is at most 46 + V / 256 in every one of these cases
(V / 64 - V / 256 is at most 30 below 2560, V / 192 - V / 256 at most 22 below 16384, V / 128 - V / 256 at most 24 below 6144),
which leaves 18 2^-24 for the factors of sums that meet a larger logit: 2^-22 each, of the part that is scaled alone, which the
larger logit makes the smaller one.  At temperature 4 an exponential is the fourth power of 2^(lz d): off by four times
(2^-22 + |lz d| 2^-24) and two roundings, 2^-20 + |l d| 2^-24 + 2^-22, where the largest logits' own, with d near 0, count most
and are exact; |l d| 2^-22 covers the rest.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_distill import check, z  # noqa: E402,F401


@pytest.mark.parametrize("V,K", [(1, 1), (29, 5), (1003, 16), (2559, 16), (2560, 16), (4099, 300), (16383, 16), (16384, 16), (20011, 400)])
@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("kw", [dict(), dict(pad=1), dict(pad=3, gpad=5), dict(inplace=True), dict(inplace=True, pad=1), dict(grad=False)])
def test_temperature_four(z, V, K, ty, kw):  # noqa: F811
    check(z, 9, V, K, ty, tau=4.0, alpha=0.5, **kw)


@pytest.mark.parametrize("V,K", [(2559, 7), (2560, 7), (6143, 0), (6144, 0), (6144, 7), (16383, 0), (16384, 0), (16383, 7), (16384, 7)])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("ty,pad,gpad", [(0, 0, 0), (1, 1, 0)])
def test_bounds_of_the_rows_lengths(z, V, K, tau, ty, pad, gpad):  # noqa: F811
    check(z, 7, V, K, ty, tau=tau, alpha=0.4, pad=pad, gpad=gpad)


@pytest.mark.parametrize("masked", [1, 900, 998])
def test_temperature_four_of_masked_rows(z, masked):  # noqa: F811
    check(z, 9, 1000, 2, 1, tau=4.0, alpha=0.7, masked=masked, twice=True)
