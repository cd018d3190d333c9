"""Refusals of the operators around the update: every argument check runs on the
host before anything is launched, so none of this needs a GPU.  Addresses are
never dereferenced."""
import ctypes as C

import pytest

A, B, S1, S2, D, W = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(6))
F = float("inf")


def _status(fn, *args):
    try:
        fn(*args)
    except Exception as e:
        return e.status
    return 0


def _gemm(hm, **kw):
    v = dict(a=A, lda=64, sa=S1, b=B, ldb=64, sb=S2, m=5, n=7, k=64, d=D, ldd=7, t=hm.HM_BF16, acc=False)
    v.update(kw)
    return _status(hm.mxfp8_gemm, *v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), "ARG"), (dict(n=-1), "ARG"), (dict(k=-32), "ARG"), (dict(a=0), "ARG"), (dict(sa=0), "ARG"),
    (dict(b=0), "ARG"), (dict(sb=0), "ARG"), (dict(d=0), "ARG"), (dict(ldd=6), "ARG"), (dict(lda=32), "ARG"),
    (dict(ldb=32), "ARG"), (dict(k=48), "ALIGN"), (dict(lda=72), "ALIGN"), (dict(ldb=72), "ALIGN"),
    (dict(a=A + 8), "ALIGN"), (dict(b=B + 1), "ALIGN"), (dict(sa=S1 + 4), "ALIGN"), (dict(sb=S2 + 4), "ALIGN"),
    (dict(d=D + 1), "ALIGN"), (dict(t=2, d=D + 2), "ALIGN"), (dict(t=0), "DTYPE"), (dict(t=3), "DTYPE"),
    (dict(acc=True), "DTYPE"), (dict(m=2 ** 31), "GEOMETRY"), (dict(lda=2 ** 31), "GEOMETRY"),
    (dict(ldd=2 ** 41), "GEOMETRY"), (dict(d=A), "OVERLAP"), (dict(d=B + 64), "OVERLAP"), (dict(d=S1), "OVERLAP"),
    (dict(d=S2 + 16), "OVERLAP"), (dict(m=0), "OK"), (dict(n=0), "OK"), (dict(m=0, d=0, a=0), "OK"),
])
def test_gemm_refusals(hm, kw, status):
    assert _gemm(hm, **kw) == (0 if status == "OK" else getattr(hm, "HM_ERR_" + status))


def _quant(hm, **kw):
    v = dict(x=A, t=hm.HM_BF16, rows=40, cols=70, ldx=70, row=0, col=0, block=32, q=B, ldq=96, s=S1, qt=D, ldqt=64,
             st=S2)
    v.update(kw)
    return _status(hm.mxfp8_quantize, *v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(cols=-1), "ARG"), (dict(block=64), "ARG"), (dict(x=0), "ARG"), (dict(ldx=69), "ARG"),
    (dict(q=0), "ARG"), (dict(s=0), "ARG"), (dict(qt=0), "ARG"), (dict(st=0), "ARG"),
    (dict(q=0, s=0, qt=0, st=0), "ARG"), (dict(ldq=80), "ARG"), (dict(ldqt=48), "ARG"), (dict(ldq=104), "ALIGN"),
    (dict(ldqt=72), "ALIGN"), (dict(x=A + 1), "ALIGN"), (dict(t=2, x=A + 2), "ALIGN"), (dict(row=W + 2), "ALIGN"),
    (dict(col=W + 1), "ALIGN"), (dict(q=B + 8), "ALIGN"), (dict(s=S1 + 8), "ALIGN"), (dict(qt=D + 8), "ALIGN"),
    (dict(st=S2 + 8), "ALIGN"), (dict(t=0), "DTYPE"), (dict(t=3), "DTYPE"), (dict(rows=2 ** 22 + 1), "GEOMETRY"),
    (dict(cols=2 ** 30 + 1), "GEOMETRY"), (dict(q=A), "OVERLAP"), (dict(qt=B), "OVERLAP"), (dict(s=S2), "OVERLAP"),
    (dict(row=S1), "OVERLAP"), (dict(rows=0), "OK"), (dict(cols=0), "OK"),
])
def test_quantize_refusals(hm, kw, status):
    assert _quant(hm, **kw) == (0 if status == "OK" else getattr(hm, "HM_ERR_" + status))


def _norm(hm, **kw):
    v = dict(x=A, ldx=64, res=B, h=D, ldh=64, t=hm.HM_BF16, rows=3, d=64, gamma=S1, eps=1e-5, block=32, rstd=W,
             q=W + 4096, s=S2)
    v.update(kw)
    return _status(hm.rmsnorm_mxfp8, *v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(d=-32), "ARG"), (dict(block=16), "ARG"), (dict(eps=-1.0), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(x=0), "ARG"), (dict(h=0), "ARG"), (dict(gamma=0), "ARG"),
    (dict(rstd=0), "ARG"), (dict(q=0), "ARG"), (dict(s=0), "ARG"), (dict(ldx=56), "ARG"), (dict(ldh=56), "ARG"),
    (dict(d=48), "ALIGN"), (dict(ldx=68), "ALIGN"), (dict(ldh=68), "ALIGN"), (dict(x=A + 8), "ALIGN"),
    (dict(res=B + 8), "ALIGN"), (dict(h=D + 8), "ALIGN"), (dict(gamma=S1 + 4), "ALIGN"), (dict(rstd=W + 2), "ALIGN"),
    (dict(q=W + 4104), "ALIGN"), (dict(s=S2 + 4), "ALIGN"), (dict(t=0), "DTYPE"),
    (dict(d=16416, ldx=16416, ldh=16416), "GEOMETRY"), (dict(rows=2 ** 31), "GEOMETRY"), (dict(h=A + 16), "OVERLAP"),
    (dict(h=A, ldh=128), "OVERLAP"), (dict(h=B + 128), "OVERLAP"), (dict(q=A), "OVERLAP"), (dict(rstd=S1), "OVERLAP"),
    (dict(s=W), "OVERLAP"), (dict(rows=0), "OK"), (dict(d=0), "OK"),
])
def test_norm_refusals(hm, kw, status):
    assert _norm(hm, **kw) == (0 if status == "OK" else getattr(hm, "HM_ERR_" + status))


def _grad(hm, **kw):
    v = dict(dy=A, lddy=64, dres=B, h=S1, dx=D, ldh=64, t=hm.HM_BF16, rows=3, d=64, gamma=S2, rstd=S2 + 4096,
             dgamma=S2 + 8192, acc=False, ws=W, ws_bytes=1 << 20)
    v.update(kw)
    return _status(hm.rmsnorm_backward, *v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(d=-32), "ARG"), (dict(dy=0), "ARG"), (dict(h=0), "ARG"), (dict(dx=0), "ARG"),
    (dict(gamma=0), "ARG"), (dict(rstd=0), "ARG"), (dict(dgamma=0), "ARG"), (dict(lddy=32), "ARG"),
    (dict(ldh=32), "ARG"), (dict(d=40), "ALIGN"), (dict(lddy=68), "ALIGN"), (dict(ldh=68), "ALIGN"),
    (dict(dy=A + 4), "ALIGN"), (dict(dres=B + 4), "ALIGN"), (dict(h=S1 + 4), "ALIGN"), (dict(dx=D + 4), "ALIGN"),
    (dict(gamma=S2 + 4), "ALIGN"), (dict(rstd=S2 + 4097), "ALIGN"), (dict(dgamma=S2 + 8193), "ALIGN"),
    (dict(ws=W + 8), "ALIGN"), (dict(t=3), "DTYPE"), (dict(d=16416), "GEOMETRY"), (dict(dx=A + 16), "OVERLAP"),
    (dict(dx=S1 + 128), "OVERLAP"), (dict(dgamma=S2), "OVERLAP"), (dict(ws=A), "OVERLAP"), (dict(ws=D), "OVERLAP"),
    (dict(dgamma=D), "OVERLAP"), (dict(d=0), "OK"),
])
def test_norm_gradient_refusals(hm, kw, status):
    assert _grad(hm, **kw) == (0 if status == "OK" else getattr(hm, "HM_ERR_" + status))


def _clip(hm, tensors, max_norm=1.0, eps=1e-6, stats=D, ws=W, ws_bytes=1 << 20):
    return _status(hm.grad_norm_clip, hm.grad_list(tensors), max_norm, eps, stats, ws, ws_bytes)


def test_clip_refusals(hm):
    good = [(A, A, 100, hm.HM_F32)]
    assert _clip(hm, good, max_norm=0.0) == hm.HM_ERR_ARG
    assert _clip(hm, good, max_norm=float("nan")) == hm.HM_ERR_ARG
    assert _clip(hm, good, eps=-1.0) == hm.HM_ERR_ARG
    assert _clip(hm, good, stats=0) == hm.HM_ERR_ARG
    assert _clip(hm, good, stats=D + 2) == hm.HM_ERR_ALIGN
    assert _clip(hm, good, ws=W + 8) == hm.HM_ERR_ALIGN
    assert _clip(hm, good, ws=0) == hm.HM_ERR_WORKSPACE
    assert _clip(hm, good, ws_bytes=0) == hm.HM_ERR_WORKSPACE
    assert _clip(hm, [(0, A, 100, hm.HM_F32)]) == hm.HM_ERR_ARG
    assert _clip(hm, [(A, A, -1, hm.HM_F32)]) == hm.HM_ERR_ARG
    assert _clip(hm, [(A, A, 100, hm.HM_U8)]) == hm.HM_ERR_DTYPE
    assert _clip(hm, [(A + 2, B, 100, hm.HM_F32)]) == hm.HM_ERR_ALIGN
    assert _clip(hm, [(A, B + 1, 100, hm.HM_BF16)]) == hm.HM_ERR_ALIGN
    assert _clip(hm, [(A, A + 4, 100, hm.HM_F32)]) == hm.HM_ERR_OVERLAP
    assert _clip(hm, [(A, A, 2 ** 43, hm.HM_F32)]) == hm.HM_ERR_GEOMETRY
    n = C.c_size_t(0)
    assert hm.lib().grad_norm_clip_workspace(None, 1, C.byref(n)) == hm.HM_ERR_ARG
    assert hm.lib().grad_norm_clip_workspace(None, 0, None) == hm.HM_ERR_ARG
    assert hm.grad_norm_clip_workspace(hm.grad_list([])) == 0


def test_size_queries(hm):
    assert hm.mxfp8_tiled_scale_bytes(0, 64) == 0
    assert hm.mxfp8_tiled_scale_bytes(1, 32) == 512
    assert hm.mxfp8_tiled_scale_bytes(129, 160) == 2 * 2 * 512
    assert _status(hm.mxfp8_tiled_scale_bytes, 1, 33) == hm.HM_ERR_ALIGN
    assert _status(hm.mxfp8_tiled_scale_bytes, -1, 32) == hm.HM_ERR_ARG
    assert hm.rmsnorm_backward_workspace(0, 64) == 0
    assert _status(hm.rmsnorm_backward_workspace, 1, 16416) == hm.HM_ERR_GEOMETRY
    assert _status(hm.rmsnorm_backward_workspace, 1, 40) == hm.HM_ERR_ALIGN
