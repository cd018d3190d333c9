"""Sizes and pitches that are each allowed but reach past any address space together:
refused on the host, before spans and offsets leave 64 bits."""
import pytest

A, B, S1, S2, D, W = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(6))
M = 2 ** 31 - 512


def _status(fn, *args):
    try:
        fn(*args)
    except Exception as e:
        return e.status
    return 0


@pytest.mark.parametrize("kw", [dict(m=M, ldd=2 ** 40), dict(m=M, lda=2 ** 30), dict(n=M, ldd=M, ldb=2 ** 30),
                                dict(m=2 ** 23 + 1, ldd=2 ** 40)])
def test_gemm(hm, kw):
    v = dict(a=A, lda=64, sa=S1, b=B, ldb=64, sb=S2, m=5, n=7, k=64, d=D, ldd=7, t=hm.HM_F32, acc=False)
    v.update(kw)
    assert _status(hm.mxfp8_gemm, *v.values()) == hm.HM_ERR_GEOMETRY


@pytest.mark.parametrize("kw", [dict(rows=2 ** 22, ldx=2 ** 40), dict(rows=2 ** 22, ldq=2 ** 40, ldqt=2 ** 22),
                                dict(cols=2 ** 30, ldx=2 ** 30, ldq=2 ** 30, ldqt=2 ** 40)])
def test_quantize(hm, kw):
    v = dict(x=A, t=hm.HM_F32, rows=40, cols=70, ldx=70, row=0, col=0, block=32, q=B, ldq=96, s=S1, qt=D, ldqt=64, st=S2)
    v.update(kw)
    assert _status(hm.mxfp8_quantize, *v.values()) == hm.HM_ERR_GEOMETRY


@pytest.mark.parametrize("kw", [dict(ldx=2 ** 40), dict(ldh=2 ** 40)])
def test_norm(hm, kw):
    v = dict(x=A, ldx=64, res=B, h=D, ldh=64, t=hm.HM_BF16, rows=M, d=64, gamma=S1, eps=1e-5, block=32, rstd=W,
             q=W + 4096, s=S2)
    v.update(kw)
    assert _status(hm.rmsnorm_mxfp8, *v.values()) == hm.HM_ERR_GEOMETRY


@pytest.mark.parametrize("kw", [dict(lddy=2 ** 40), dict(ldh=2 ** 40)])
def test_norm_gradient(hm, kw):
    v = dict(dy=A, lddy=64, dres=B, h=S1, dx=D, ldh=64, t=hm.HM_BF16, rows=M, d=64, gamma=S2, rstd=S2 + 4096,
             dgamma=S2 + 8192, acc=False, ws=W, ws_bytes=1 << 20)
    v.update(kw)
    assert _status(hm.rmsnorm_backward, *v.values()) == hm.HM_ERR_GEOMETRY
