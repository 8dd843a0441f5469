"""A wait of AdamW's pipeline that runs out, without a GPU fault: the diagnostic's first CTA never hands a stage of its ring
back, and the lanes of its copying warp get different answers.  They have to give up together, count one timeout and
return; the context stays usable for the next step."""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HYPER = (1e-2, 0.9, 0.999, 1e-8)


@pytest.fixture(scope="module")
def z(zlib):
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    return zlib


def make(z, n, bits=32, gt=0):
    gen = torch.Generator(device="cuda").manual_seed(n)
    t = dict(grad=torch.randn(n, generator=gen, device="cuda").to((torch.float16, torch.bfloat16)[gt]),
             master=torch.randn(n, generator=gen, device="cuda"), param=torch.empty(n, dtype=torch.float16, device="cuda"), n=n)
    if bits == 32:
        t.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
    else:
        t.update(m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 m_scale=torch.zeros(n // 256 + 1, device="cuda"), v_scale=torch.zeros(n // 256 + 1, device="cuda"))
    return t, z.zero_adamw_plan([t], 1, gt, 0, bits)


def test_the_copying_warp_gives_up_together(z):
    n = 4096 * 2048 + 5000
    start, plan = make(z, n)
    assert plan.info.pipeline == 1 and z.zero_train_timeouts(reset=True) >= 0
    want, other = make(z, n)
    z.zero_adamw_step(other, None, 1, *HYPER)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    z.zero_selftest_adamw_wait(plan, 1, *HYPER)
    torch.cuda.synchronize()
    elapsed = time.monotonic() - t0
    assert z.zero_train_timeouts(reset=True) == 1
    assert 1.5 < elapsed < 60, elapsed
    # the other CTAs' elements are those of the step, the first one's chunks after its ring's are as they were
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunk = torch.arange(n, device="cuda") // 2048
    others = chunk % sms != 0
    for key in ("master", "m", "v"):
        assert torch.equal(start[key][others], want[key][others]), key
    late = ~others & (chunk // sms >= 15)
    assert bool(late.any()) and not start["m"][late].any() and not start["v"][late].any()
    # the context still works: the same step from the same state
    again, plan = make(z, n)
    z.zero_adamw_step(plan, None, 1, *HYPER)
    for key in ("master", "m", "v", "param"):
        assert torch.equal(again[key], want[key]), key
    assert z.zero_train_timeouts() == 0


def test_the_diagnostic_refuses_other_plans(z):
    for n, bits, gt in ((100000, 32, 0), (4096 * 2048, 8, 0), (4096 * 2048, 32, 1)):
        t, plan = make(z, n, bits, gt)
        was = t["master"].clone()
        with pytest.raises(z.ZeroError) as e:
            z.zero_selftest_adamw_wait(plan, 1, *HYPER)
        assert e.value.code == z.ZERO_EINVAL
        torch.cuda.synchronize()
        assert torch.equal(t["master"], was)
    assert z.zero_train_timeouts() == 0
