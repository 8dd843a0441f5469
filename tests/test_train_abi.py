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


def test_linear_workspace(zlib):
    z = zlib
    assert z.zero_linear_workspace(100, 64, 128, 0, False, True) == 0
    assert z.zero_linear_workspace(100, 63, 128, 0, False, False) >= (100 + 128) * 64 * 2
    assert z.zero_linear_workspace(100, 64, 128, 2, True, True) >= 100 * 128 * 2 + 128 * 4
    for args in [(-1, 64, 128, 0), (1, 0, 128, 0), (1, 64, 0, 0), (1, 64, 128, 4), (1 << 31, 64, 64, 0), (1 << 30, 1 << 30, 1, 0)]:
        with pytest.raises(z.ZeroError) as e:
            z.zero_linear_workspace(*args, False, True)
        assert e.value.code == z.ZERO_EINVAL


X, W, B, Y, ZZ, DX, DW, DB, DY, WS = (BASE * (16 + 16 * k) for k in range(10))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(T=-1), -1), (dict(K=0), -1), (dict(N=1 << 31), -1), (dict(ldx=63), -1),
    (dict(ldw=63), -1), (dict(ldy=127), -1), (dict(z=ZZ, ldz=100), -1), (dict(r=ZZ, ldr=100), -1), (dict(act=5), -1), (dict(ty=2), -1),
    (dict(x=X + 2), -1), (dict(ldw=65), -1), (dict(x=X + 2, ws=WS, n=100), -1), (dict(x=X + 2, ws=WS + 8, n=1 << 20), -2), (dict(x=X + 2, ws=Y - 256, n=1 << 20), -3),
    (dict(x=X + 1), -2), (dict(b=B + 1), -2), (dict(y=Y + 1), -2),
    (dict(y=X), -3), (dict(y=W + 64), -3), (dict(y=B), -3), (dict(z=Y + 2, ldz=128), -3), (dict(r=Y + 2, ldr=128), -3), (dict(z=B, ldz=128), -3)])
def test_linear_forward_refuses(zlib, kw, code):
    a = dict(x=X, ldx=64, w=W, ldw=64, b=B, r=None, ldr=0, y=Y, ldy=128, z=None, ldz=0, T=10, K=64, N=128, act=0, ty=0, ws=None, n=0)
    a.update(kw)
    assert zlib.lib().zero_linear_forward(*a.values(), None) == code


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(z=None), -1), (dict(dx=None, dw=None, db=None), -1), (dict(lddy=100), -1),
    (dict(ldz=100), -1), (dict(lddx=60), -1), (dict(lddw=60), -1), (dict(act=9), -1), (dict(ty=2), -1), (dict(ws=None, n=0), -1), (dict(n=100), -1),
    (dict(dy=DY + 1), -2), (dict(dw=DW + 1), -2), (dict(db=DB + 1), -2), (dict(ws=WS + 4), -2),
    (dict(dx=DY), -3), (dict(dw=X), -3), (dict(db=DW + 64), -3), (dict(dw=DX + 64), -3), (dict(dx=W), -3), (dict(db=ZZ), -3), (dict(ws=DX), -3), (dict(ws=ZZ + 256), -3)])
def test_linear_backward_refuses(zlib, kw, code):
    a = dict(dy=DY, lddy=128, z=ZZ, ldz=128, x=X, ldx=64, w=W, ldw=64, dx=DX, lddx=64, dw=DW, lddw=64, db=DB, T=10, K=64, N=128, act=2, ty=0,
             ws=WS, n=1 << 20)
    a.update(kw)
    assert zlib.lib().zero_linear_backward(*a.values(), None) == code
