"""include/zero_train.h without a GPU: the header as strict C11, the plan of an
AdamW step (host only), and the refusals that come before any CUDA call."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

from conftest import ROOT, cuda_available

no_gpu = pytest.mark.skipif(cuda_available(), reason="made-up addresses: only where no kernel can run")
BASE = 1 << 20


def rows(z, count, **kw):
    arr = (z.zero_adamw_tensor_t * count)()
    for j in range(count):
        a, o = arr[j], BASE * 64 * (j + 1)
        a.n, a.rank_stride, a.lr_scale, a.weight_decay = 1000, 1000, 1.0, 0.0
        for k, key in enumerate(("grad", "master", "m", "v", "param", "m_scale", "v_scale")):
            setattr(a, key, o + k * BASE)
    for key, value in kw.items():
        setattr(arr[0], key, value)
    return arr


def plan(z, arr, P=1, gt=0, pt=0, bits=32, table=None, cap=0):
    info = z.zero_adamw_plan_t()
    rc = z.lib().zero_adamw_plan(arr, len(arr), P, gt, pt, bits, ctypes.byref(info), table, cap)
    return rc, info


def test_header_is_strict_c11(tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no gcc")
    src = tmp_path / "t.c"
    src.write_text('#include "zero_train.h"\nint main(void) { zero_adamw_plan_t p; (void)p; return 0; }\n')
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def test_plan_counts(zlib):
    z = zlib
    rc, info = plan(z, rows(z, 3))
    assert rc == 0 and info.elements == 3000 and info.chunks == 3 and info.vector_tensors == 3
    table = (ctypes.c_ubyte * info.table_bytes)()
    assert plan(z, rows(z, 3), table=table, cap=info.table_bytes)[0] == 0
    assert plan(z, rows(z, 3), table=table, cap=info.table_bytes - 1)[0] == z.ZERO_EINVAL
    # an empty tensor has no chunk and needs no buffer
    arr = rows(z, 2, n=0, grad=None, master=None, m=None, v=None, param=None)
    rc, info = plan(z, arr)
    assert rc == 0 and info.elements == 1000 and info.chunks == 1
    # streams on another phase than the parameters go element by element
    assert plan(z, rows(z, 1, master=BASE * 65 + 4))[1].vector_tensors == 0
    # all streams 3 elements in: 32-bit moments keep whole vectors, 8-bit ones (whose scales start with the tensor) do not
    o = BASE * 64
    off = dict(grad=o + 6, master=o + BASE + 12, m=o + 2 * BASE + 12, v=o + 3 * BASE + 12, param=o + 4 * BASE + 6)
    assert plan(z, rows(z, 1, **off))[1].vector_tensors == 1
    off.update(m=o + 2 * BASE + 3, v=o + 3 * BASE + 3)
    assert plan(z, rows(z, 1, **off), bits=8)[1].vector_tensors == 0


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(grad=None), -1), (dict(master=None), -1), (dict(m=None), -1), (dict(v=None), -1),
    (dict(param=None), -1), (dict(weight_decay=-1.0), -1), (dict(weight_decay=math.inf), -1), (dict(lr_scale=math.nan), -1),
    (dict(grad=BASE * 64 + 1), -2), (dict(master=BASE * 65 + 2), -2), (dict(m=BASE * 66 + 1), -2), (dict(param=BASE * 68 + 1), -2),
    (dict(m=BASE * 65 + 3996), -3), (dict(param=BASE * 64 + 1998), -3), (dict(v=BASE * 129), -3)])
def test_plan_refuses(zlib, kw, code):
    arr = rows(zlib, 2, **kw)
    info = zlib.zero_adamw_plan_t(n_tensors=77)
    assert zlib.lib().zero_adamw_plan(arr, 2, 1, 0, 0, 32, ctypes.byref(info), None, 0) == code
    assert info.n_tensors == 77                       # a refused call leaves the plan as it was


def test_plan_refuses_scalars(zlib):
    z = zlib
    for kw in (dict(P=0), dict(P=1025), dict(gt=3), dict(gt=-1), dict(pt=2), dict(bits=16)):
        assert plan(z, rows(z, 1), **kw)[0] == z.ZERO_EINVAL, kw
    assert plan(z, rows(z, 1, rank_stride=999), P=2)[0] == z.ZERO_EINVAL
    assert plan(z, rows(z, 1, rank_stride=999), P=1)[0] == z.ZERO_OK
    assert plan(z, rows(z, 1, m_scale=None), bits=8)[0] == z.ZERO_EINVAL
    assert plan(z, rows(z, 1, m_scale=BASE * 68), bits=8)[0] == z.ZERO_EOVERLAP
    assert plan(z, rows(z, 1, master=None, m=None, v=None, param=None), bits=0, pt=9)[0] == z.ZERO_OK
    # a written buffer between two ranks' gradients is fine, one inside a rank's is not
    assert plan(z, rows(z, 1, rank_stride=BASE * 8, master=BASE * 64 + 4000), P=2)[0] == z.ZERO_OK
    assert plan(z, rows(z, 1, rank_stride=4000, master=BASE * 64 + 8000), P=2)[0] == z.ZERO_EOVERLAP


@no_gpu
def test_step_and_norm_refuse(zlib):
    z = zlib
    L = z.lib()
    _, info = plan(z, rows(z, 1))
    ok = dict(t=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8)
    for kw in (dict(t=0), dict(lr=math.nan), dict(b1=1.0), dict(b2=-0.1), dict(eps=-1.0), dict(eps=math.inf)):
        a = dict(ok, **kw)
        assert L.zero_adamw_step(ctypes.byref(info), BASE, None, a["t"], a["lr"], a["b1"], a["b2"], a["eps"], 0, None) == z.ZERO_EINVAL
    assert L.zero_adamw_step(ctypes.byref(info), None, None, 1, 1e-3, 0.9, 0.999, 1e-8, 0, None) == z.ZERO_EINVAL
    assert L.zero_adamw_step(ctypes.byref(info), BASE + 8, None, 1, 1e-3, 0.9, 0.999, 1e-8, 0, None) == z.ZERO_EALIGN
    for scale, top in ((0.0, 1.0), (-1.0, 1.0), (math.nan, 1.0), (1.0, math.nan)):
        assert L.zero_grad_norm(ctypes.byref(info), BASE, scale, top, BASE * 2, None) == z.ZERO_EINVAL
    assert L.zero_grad_norm(ctypes.byref(info), BASE, 1.0, 1.0, None, None) == z.ZERO_EINVAL
    assert L.zero_grad_norm(ctypes.byref(info), BASE, 1.0, 1.0, BASE + 2, None) == z.ZERO_EALIGN
    _, grads_only = plan(z, rows(z, 1), bits=0)
    assert L.zero_adamw_step(ctypes.byref(grads_only), BASE, None, 1, 1e-3, 0.9, 0.999, 1e-8, 0, None) == z.ZERO_EINVAL
