"""What the layers' entry points refuse before any CUDA call (made-up addresses: only where no kernel can run), and their
workspaces."""
import math

import pytest

from conftest import cuda_available

no_gpu = pytest.mark.skipif(cuda_available(), reason="made-up addresses: only where no kernel can run")
M = 1 << 24
A, B, C, D, E, F, G, H, I, J, K, WS = (M * (k + 1) for k in range(12))
E_INVAL, E_ALIGN, E_OVERLAP, E_CUDA = -1, -2, -3, -4


def call(zlib, name, order, base, kw):
    a = dict(base)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(zlib.lib(), name)(*(a[k] for k in order.split()), None)


EMBED = ("zero_embed_forward", "ids table ldt y ldy T D V scale type", dict(ids=A, table=B, ldt=64, y=C, ldy=64, T=10, D=64, V=100, scale=1.0, type=0))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(), E_CUDA), (dict(T=0, ids=None, table=None, y=None), 0), (dict(ids=None), E_INVAL), (dict(table=None), E_INVAL), (dict(y=None), E_INVAL), (dict(T=-1), E_INVAL),
    (dict(D=0), E_INVAL), (dict(V=0), E_INVAL), (dict(V=(1 << 30) + 1), E_INVAL), (dict(D=(1 << 30) + 1), E_INVAL), (dict(T=1 << 31), E_INVAL), (dict(ldt=63), E_INVAL),
    (dict(ldy=63), E_INVAL), (dict(scale=math.inf), E_INVAL), (dict(scale=math.nan), E_INVAL), (dict(type=2), E_INVAL), (dict(type=-1), E_INVAL),
    (dict(ids=A + 2), E_ALIGN), (dict(table=B + 1), E_ALIGN), (dict(y=C + 1), E_ALIGN), (dict(y=B + 64), E_OVERLAP), (dict(y=A), E_OVERLAP)])
def test_embed_forward(zlib, kw, code):
    assert call(zlib, *EMBED, kw) == code


EMBED_BACK = ("zero_embed_backward", "ids dy lddy dt lddt T D V scale add type ws n",
              dict(ids=A, dy=B, lddy=64, dt=C, lddt=64, T=10, D=64, V=100, scale=1.0, add=0, type=0, ws=WS, n=1 << 22))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(), E_CUDA), (dict(T=0, add=1, ids=None, dy=None, ws=None, n=0), 0), (dict(ids=None), E_INVAL), (dict(dy=None), E_INVAL), (dict(dt=None), E_INVAL),
    (dict(dt=None, T=0), E_INVAL), (dict(T=-1), E_INVAL), (dict(D=0), E_INVAL), (dict(V=0), E_INVAL), (dict(lddy=63), E_INVAL), (dict(lddt=63), E_INVAL),
    (dict(scale=-math.inf), E_INVAL), (dict(type=2), E_INVAL), (dict(ws=None), E_INVAL), (dict(n=100), E_INVAL), (dict(ws=WS + 8), E_ALIGN), (dict(ids=A + 1), E_ALIGN),
    (dict(dy=B + 1), E_ALIGN), (dict(dt=C + 1), E_ALIGN), (dict(dt=B + 64), E_OVERLAP), (dict(dt=A), E_OVERLAP), (dict(ws=A), E_OVERLAP), (dict(ws=B - 256), E_OVERLAP),
    (dict(ws=C - 256), E_OVERLAP)])
def test_embed_backward(zlib, kw, code):
    assert call(zlib, *EMBED_BACK, kw) == code


NORM = ("zero_layernorm_forward", "x ldx w b y ldy mean rstd T D eps type",
        dict(x=A, ldx=64, w=B, b=C, y=D, ldy=64, mean=E, rstd=F, T=10, D=64, eps=1e-5, type=0))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(), E_CUDA), (dict(w=None, b=None, mean=None, rstd=None), E_CUDA), (dict(y=A), E_CUDA), (dict(T=0, x=None, y=None), 0), (dict(x=None), E_INVAL),
    (dict(y=None), E_INVAL), (dict(T=-1), E_INVAL), (dict(D=0), E_INVAL), (dict(D=(1 << 30) + 1), E_INVAL), (dict(ldx=63), E_INVAL), (dict(ldy=63), E_INVAL),
    (dict(eps=0.0), E_INVAL), (dict(eps=-1.0), E_INVAL), (dict(eps=math.nan), E_INVAL), (dict(eps=math.inf), E_INVAL), (dict(eps=1e-40), E_INVAL), (dict(type=2), E_INVAL),
    (dict(x=A + 1), E_ALIGN), (dict(w=B + 1), E_ALIGN), (dict(b=C + 1), E_ALIGN), (dict(y=D + 1), E_ALIGN), (dict(mean=E + 2), E_ALIGN), (dict(rstd=F + 2), E_ALIGN),
    (dict(y=A + 2), E_OVERLAP), (dict(y=A, ldy=72), E_OVERLAP), (dict(y=B), E_OVERLAP), (dict(y=C), E_OVERLAP), (dict(rstd=E + 36), E_OVERLAP), (dict(mean=A), E_OVERLAP),
    (dict(mean=D + 4), E_OVERLAP), (dict(rstd=B), E_OVERLAP), (dict(rstd=C), E_OVERLAP)])
def test_layernorm_forward(zlib, kw, code):
    assert call(zlib, *NORM, kw) == code


NORM_BACK = ("zero_layernorm_backward", "dy lddy x ldx w mean rstd res ldr dx lddx dw db T D type ws n",
             dict(dy=A, lddy=64, x=B, ldx=64, w=C, mean=D, rstd=E, res=F, ldr=64, dx=G, lddx=64, dw=H, db=I, T=10, D=64, type=0, ws=WS, n=1 << 22))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(), E_CUDA), (dict(res=None, w=None), E_CUDA), (dict(dx=F), E_CUDA), (dict(dx=A), E_CUDA), (dict(dw=None, db=None, ws=None, n=0), E_CUDA),
    (dict(dx=None, dw=None, db=None), E_INVAL), (dict(dy=None), E_INVAL), (dict(x=None), E_INVAL), (dict(mean=None), E_INVAL), (dict(rstd=None), E_INVAL), (dict(T=-1), E_INVAL),
    (dict(D=0), E_INVAL), (dict(lddy=63), E_INVAL), (dict(ldx=63), E_INVAL), (dict(ldr=63), E_INVAL), (dict(lddx=63), E_INVAL), (dict(type=2), E_INVAL), (dict(ws=None), E_INVAL),
    (dict(n=100), E_INVAL), (dict(ws=WS + 8), E_ALIGN), (dict(dy=A + 1), E_ALIGN), (dict(dx=G + 1), E_ALIGN), (dict(mean=D + 2), E_ALIGN), (dict(dw=H + 1), E_ALIGN),
    (dict(dx=B), E_OVERLAP), (dict(dx=A + 2), E_OVERLAP), (dict(dx=A, D=17000, lddx=17000, lddy=17000, ldx=17000, ldr=17000, n=1 << 23), E_OVERLAP), (dict(dw=A), E_OVERLAP),
    (dict(db=H + 64), E_OVERLAP), (dict(dw=G), E_OVERLAP), (dict(dw=C), E_OVERLAP), (dict(db=D), E_OVERLAP), (dict(ws=A), E_OVERLAP), (dict(ws=G - 256), E_OVERLAP)])
def test_layernorm_backward(zlib, kw, code):
    assert call(zlib, *NORM_BACK, kw) == code


GATED = ("zero_gated_forward", "x ldx wg ldg_ wu ldu_ bg bu h ldh g ldg u ldu T K N act type ws n",
         dict(x=A, ldx=64, wg=B, ldg_=64, wu=C, ldu_=64, bg=D, bu=E, h=F, ldh=128, g=G, ldg=128, u=H, ldu=128, T=10, K=64, N=128, act=3, type=0, ws=None, n=0))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(T=0, x=None, h=None), 0), (dict(x=None), E_INVAL), (dict(wg=None), E_INVAL), (dict(wu=None), E_INVAL), (dict(h=None), E_INVAL), (dict(g=None), E_INVAL), (dict(u=None), E_INVAL),
    (dict(T=-1), E_INVAL), (dict(K=0), E_INVAL), (dict(N=0), E_INVAL), (dict(N=1 << 30), E_INVAL), (dict(ldx=63), E_INVAL), (dict(ldg_=63), E_INVAL), (dict(ldu_=63), E_INVAL),
    (dict(ldh=127), E_INVAL), (dict(ldg=127), E_INVAL), (dict(ldu=127), E_INVAL), (dict(act=4), E_INVAL), (dict(act=-1), E_INVAL), (dict(type=2), E_INVAL), (dict(x=A + 2), E_INVAL),
    (dict(x=A + 2, ws=WS, n=64), E_INVAL), (dict(x=A + 2, ws=WS + 8, n=1 << 22), E_ALIGN), (dict(x=A + 2, ws=F - 256, n=1 << 22), E_OVERLAP), (dict(wu=C + 1), E_ALIGN),
    (dict(h=F + 1), E_ALIGN), (dict(bu=E + 1), E_ALIGN), (dict(h=A), E_OVERLAP), (dict(h=B + 64), E_OVERLAP), (dict(g=C), E_OVERLAP), (dict(g=F + 2), E_OVERLAP), (dict(u=G + 64), E_OVERLAP),
    (dict(u=D), E_OVERLAP)])
def test_gated_forward(zlib, kw, code):
    assert call(zlib, *GATED, kw) == code


GATED_BACK = ("zero_gated_backward", "dh lddh g ldg u ldu x ldx wg ldg_ wu ldu_ dx lddx dwg lddwg dwu lddwu dbg dbu T K N act type ws n",
              dict(dh=A, lddh=128, g=B, ldg=128, u=C, ldu=128, x=D, ldx=64, wg=E, ldg_=64, wu=F, ldu_=64, dx=G, lddx=64, dwg=H, lddwg=64, dwu=I, lddwu=64, dbg=J, dbu=K,
                   T=10, K=64, N=128, act=3, type=0, ws=WS, n=1 << 22))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(dx=None, dwg=None, dwu=None, dbg=None, dbu=None), E_INVAL), (dict(dh=None), E_INVAL), (dict(g=None), E_INVAL), (dict(u=None), E_INVAL), (dict(x=None), E_INVAL),
    (dict(wg=None), E_INVAL), (dict(wu=None), E_INVAL), (dict(lddh=127), E_INVAL), (dict(ldg=127), E_INVAL), (dict(ldu=127), E_INVAL), (dict(ldx=63), E_INVAL), (dict(ldg_=63), E_INVAL),
    (dict(lddx=63), E_INVAL), (dict(lddwg=63), E_INVAL), (dict(lddwu=63), E_INVAL), (dict(lddwu=63, T=0), E_INVAL), (dict(act=9), E_INVAL), (dict(type=2), E_INVAL), (dict(ws=None), E_INVAL),
    (dict(n=100), E_INVAL), (dict(ws=WS + 4), E_ALIGN), (dict(dh=A + 1), E_ALIGN), (dict(dwu=I + 1), E_ALIGN), (dict(dbu=K + 1), E_ALIGN), (dict(dx=A), E_OVERLAP), (dict(dwg=D), E_OVERLAP),
    (dict(dwu=H + 64), E_OVERLAP), (dict(dwg=G), E_OVERLAP), (dict(dx=E), E_OVERLAP), (dict(dbg=B), E_OVERLAP), (dict(dbu=J + 64), E_OVERLAP), (dict(ws=G), E_OVERLAP), (dict(ws=C - 256), E_OVERLAP)])
def test_gated_backward(zlib, kw, code):
    assert call(zlib, *GATED_BACK, kw) == code


LOSS = ("zero_distill_loss", "logits ldl targets index teacher ldk weights loss grad ldg T V K z alpha scale type tt",
        dict(logits=A, ldl=100, targets=B, index=C, teacher=D, ldk=8, weights=E, loss=F, grad=G, ldg=100, T=10, V=100, K=8, z=2.0, alpha=0.5, scale=1.0, type=0, tt=2))


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(), E_CUDA), (dict(grad=A), E_CUDA), (dict(grad=None, weights=None), E_CUDA), (dict(alpha=0.0, index=None, teacher=None, tt=9, ldk=0), E_CUDA),
    (dict(alpha=1.0, targets=None), E_CUDA), (dict(K=0, index=None, teacher=None), E_CUDA), (dict(T=0, logits=None, loss=None), 0),
    (dict(logits=None), E_INVAL), (dict(loss=None), E_INVAL), (dict(targets=None), E_INVAL), (dict(index=None), E_INVAL), (dict(teacher=None), E_INVAL), (dict(T=-1), E_INVAL),
    (dict(V=0), E_INVAL), (dict(V=(1 << 30) + 1, ldl=1 << 31, ldg=1 << 31), E_INVAL), (dict(K=-1), E_INVAL), (dict(K=1025, ldk=1025), E_INVAL), (dict(ldl=99), E_INVAL), (dict(ldg=99), E_INVAL),
    (dict(ldk=7), E_INVAL), (dict(z=0.0), E_INVAL), (dict(z=2000.0), E_INVAL), (dict(z=math.nan), E_INVAL), (dict(alpha=-0.1), E_INVAL), (dict(alpha=1.1), E_INVAL), (dict(alpha=math.nan), E_INVAL),
    (dict(scale=math.inf), E_INVAL), (dict(type=2), E_INVAL), (dict(tt=3), E_INVAL),
    (dict(logits=A + 1), E_ALIGN), (dict(targets=B + 2), E_ALIGN), (dict(index=C + 2), E_ALIGN), (dict(teacher=D + 2), E_ALIGN), (dict(weights=E + 2), E_ALIGN), (dict(loss=F + 2), E_ALIGN),
    (dict(grad=G + 1), E_ALIGN), (dict(grad=A + 2), E_OVERLAP), (dict(grad=A, ldg=104), E_OVERLAP), (dict(loss=A), E_OVERLAP), (dict(loss=B), E_OVERLAP), (dict(loss=C + 64), E_OVERLAP),
    (dict(loss=D), E_OVERLAP), (dict(loss=E), E_OVERLAP), (dict(loss=G + 100), E_OVERLAP), (dict(grad=B - 4), E_OVERLAP), (dict(grad=D - 64), E_OVERLAP)])
def test_distill_loss(zlib, kw, code):
    assert call(zlib, *LOSS, kw) == code


def test_teacher_in_16_bits_may_lie_on_two_bytes(zlib):
    if cuda_available():
        pytest.skip("made-up addresses")
    assert call(zlib, *LOSS, dict(teacher=D + 2, tt=0)) == E_CUDA


def test_workspaces(zlib):
    z = zlib
    assert z.zero_embed_workspace(0, 64, 100) == 0 and z.zero_layernorm_workspace(0, 64) == 0
    assert z.zero_embed_workspace(10, 64, 100) >= 80 and z.zero_layernorm_workspace(10, 64) >= 2 * 64 * 4
    assert z.zero_gated_workspace(100, 64, 128, False, True) == 0
    assert z.zero_gated_workspace(100, 63, 128, False, False) >= (100 + 256) * 64 * 2
    assert z.zero_gated_workspace(100, 64, 130, True, True) >= 100 * 2 * 192 * 2 + 2 * 130 * 4
    # about a quarter of dy's elements in fp32 for the parts of runs, more for few tokens only
    assert z.zero_embed_workspace(1 << 20, 2048, 50000) < (1 << 20) * (2048 // 4 + 64)
    for f, args in ((z.zero_embed_workspace, (-1, 64, 100)), (z.zero_embed_workspace, (1, 0, 100)), (z.zero_embed_workspace, (1, 64, 0)),
                    (z.zero_layernorm_workspace, (-1, 64)), (z.zero_layernorm_workspace, (1, 0)), (z.zero_layernorm_workspace, (1, 1 << 31)),
                    (z.zero_gated_workspace, (-1, 64, 64, False, True)), (z.zero_gated_workspace, (1, 0, 64, False, True)), (z.zero_gated_workspace, (1, 64, 1 << 30, True, True))):
        with pytest.raises(z.ZeroError) as e:
            f(*args)
        assert e.value.code == z.ZERO_EINVAL
