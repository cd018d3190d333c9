"""The operators around the update against the float64 oracle, through the C ABI.

Tolerances (fixed by derivation, u = 2^-24):
  product    fp32 accumulation: each of the K/32 tensor-core steps may lose one
             unit in the last place of the running sum, and each of its 32
             addends one of the largest: (K/32 + 33) 2u of sum |a b|; a bf16
             output adds half a bf16 ulp (8 significant bits), 2^-8 |D|, an
             accumulated one 2u |D|.
  quantize   bit-exact: the fp32 products are in a stated order.
  norm       h bit-exact; rstd: the sum of squares runs through at most 8 V + 5
             + 16 additions in a row (V <= 4 vectors per thread), so 53 u
             relative, half of that after the root, plus 4 roundings: 32 u;
             the codes bit-exact given the kernel's own rstd.
  gradient   dx: the same chain for the mean, and 8 roundings of each term:
             64 u (|dres| + rstd (|t| + |xhat| mean |t xhat|)), plus 2^-8 |dx|
             for bf16; dgamma: rows + 64 additions: (rows + 64) u sum |dy xhat|.
  clip       norm 4 u relative (double sums of 128-term fp32 sums: 128 u would
             be the bound of a chain, but every term is rounded once in an fma
             chain of at most 128: 128 u); outputs bit-exact given the
             kernel's coefficient.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mxfp8 as OX  # noqa: E402
from oracle import operators as OO  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _up(x, k):
    return -(-x // k) * k


def _dt(hm, name):
    return (torch.bfloat16, hm.HM_BF16) if name == "bf16" else (torch.float32, hm.HM_F32)


def _np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _spread(rng, rows, k):
    """Gaussian values times a power of two 2^-6 .. 2^6 per 32 columns of each row."""
    e = np.repeat(rng.integers(-6, 7, (rows, _up(k, 32) // 32)), 32, axis=1)[:, :k]
    return (rng.standard_normal((rows, k)) * 0.05 * np.ldexp(1.0, e)).astype(np.float32)


def _operand(dev, rng, rows, k, block, extra=0):
    """Codes and scales on the host and on the device; the device's pitch padding holds
    NaN codes and the tiled layout's padding NaN scales, neither of which may matter."""
    codes, sf = OO.quantize(_spread(rng, rows, k), block)
    wide = np.full((rows, k + extra), 0x7F, dtype=np.uint8)
    wide[:, :k] = codes
    real = OX.scale_tile_128x4(np.ones_like(sf)) == 1
    tiled = np.where(real, OX.scale_tile_128x4(sf), 0xFF).astype(np.uint8)
    return codes, sf, torch.from_numpy(wide).to(dev), torch.from_numpy(tiled).to(dev)


def _gemm(hm, qa, ta, qb, tb, m, n, k, d, acc=False, stream=0):
    hm.mxfp8_gemm(qa.data_ptr(), qa.shape[1], ta.data_ptr(), qb.data_ptr(), qb.shape[1], tb.data_ptr(), m, n, k,
                  d.data_ptr(), d.shape[1], hm.HM_F32 if d.dtype == torch.float32 else hm.HM_BF16, acc, stream)


def _check_product(d, ref, bound, k, bf16, prior=None):
    tol = (k / 32 + 33) * 2 * U * bound
    if prior is not None:
        ref = ref + prior
        tol = tol + 2 * U * np.abs(ref)
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(_np64(d) - ref)
    assert np.isfinite(err).all()
    assert (err <= tol + 1e-37).all(), f"worst excess {np.max(err / (tol + 1e-37))}"


GEMM = [
    # m, n, k, block, out, accumulate, ldd - n, lda - k
    (1, 1, 32, 32, "f32", False, 0, 0),
    (1, 5120, 5120, 32, "bf16", False, 0, 0),
    (1, 129, 96, 128, "bf16", False, 1, 0),
    (2, 1408, 2048, 32, "f32", True, 0, 16),
    (16, 128, 1024, 32, "bf16", False, 8, 0),
    (17, 130, 160, 128, "f32", False, 3, 0),
    (33, 257, 416, 32, "bf16", False, 0, 32),
    (64, 64, 64, 32, "f32", False, 0, 0),
    (65, 320, 4128, 32, "bf16", False, 5, 0),
    (77, 1408, 2048, 128, "bf16", False, 0, 0),
    (128, 300, 4096, 32, "f32", True, 0, 0),
    (129, 256, 128, 32, "bf16", False, 0, 0),
    (130, 255, 32, 32, "f32", False, 1, 0),
    (257, 511, 224, 128, "bf16", False, 0, 16),
    (300, 700, 1056, 32, "f32", True, 4, 0),
    (513, 1030, 640, 32, "bf16", False, 2, 0),
    (1000, 1024, 2080, 128, "f32", False, 0, 0),
    (3000, 2600, 544, 32, "bf16", False, 0, 0),   # several tiles per CTA of the persistent kernel
]


@pytest.mark.parametrize("m,n,k,block,out,acc,pad,extra", GEMM)
def test_product(hm, dev, m, n, k, block, out, acc, pad, extra):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, sa, qa, ta = _operand(dev, rng, m, k, block, extra)
    b, sb, qb, tb = _operand(dev, rng, n, k, block, extra)
    dt, _ = _dt(hm, out)
    ref, bound = OO.product(a, sa, b, sb)
    prior = rng.standard_normal((m, n)).astype(np.float32) if acc else None
    d = torch.full((m + 1, n + pad), 7.0, dtype=dt, device=dev)
    if acc:
        d[:m, :n] = torch.from_numpy(prior).to(dev)
    _gemm(hm, qa, ta, qb, tb, m, n, k, d, acc)
    torch.cuda.synchronize()
    assert hm.hm_device_error() == 0
    _check_product(d[:m, :n], ref, bound, k, out == "bf16", prior)
    assert (d[m:] == 7.0).all() and (d[:, n:] == 7.0).all()   # nothing outside m x n is written
    if not acc:   # the same bits every time
        again = torch.zeros_like(d)
        _gemm(hm, qa, ta, qb, tb, m, n, k, again)
        assert torch.equal(again[:m, :n], d[:m, :n])


def test_product_offset_views_and_column_major_strides(hm, dev):
    """Operands and D inside larger allocations: a row slice of A, a column slice of D that
    is aligned to its element only."""
    rng = np.random.default_rng(8)
    m, n, k = 40, 72, 96
    a, sa, qa, ta = _operand(dev, rng, m, k, 32)
    b, sb, qb, tb = _operand(dev, rng, n, k, 32)
    big = torch.full((m + 3, 160), 0x7F, dtype=torch.uint8, device=dev)
    big[3:, 32:128] = qa
    ref, bound = OO.product(a, sa, b, sb)
    for rows, dt, code in ((m, torch.bfloat16, hm.HM_BF16), (m, torch.float32, hm.HM_F32)):
        d = torch.full((rows, 201), 5.0, dtype=dt, device=dev)
        view = d[:, 3:3 + n]
        hm.mxfp8_gemm(big[3:, 32:].data_ptr(), 160, ta.data_ptr(), qb.data_ptr(), k, tb.data_ptr(), m, n, k,
                      view.data_ptr(), 201, code)
        torch.cuda.synchronize()
        _check_product(view, ref, bound, k, dt == torch.bfloat16)
        assert (d[:, :3] == 5.0).all() and (d[:, 3 + n:] == 5.0).all()


@pytest.mark.parametrize("m", [3, 200])
def test_product_empty_sums_nan_and_zero_blocks(hm, dev, m):
    rng = np.random.default_rng(m)
    n, k = 140, 64
    a, sa, qa, ta = _operand(dev, rng, m, k, 32)
    b, sb, qb, tb = _operand(dev, rng, n, k, 32)
    d = torch.full((m, n), 3.0, device=dev)
    hm.mxfp8_gemm(0, 0, 0, 0, 0, 0, m, n, 0, d.data_ptr(), n, hm.HM_F32, True)
    assert (d == 3.0).all()
    hm.mxfp8_gemm(0, 0, 0, 0, 0, 0, m, n, 0, d.data_ptr(), n, hm.HM_F32, False)
    assert (d == 0.0).all()
    # a NaN code spoils its row, a NaN scale its column, a zero block nothing
    qa[1, 5] = 0x7F
    qb[2, :32] = 0
    at = int(np.nonzero(OX.scale_tile_128x4(np.eye(n, k // 32, dtype=np.uint8)[::1]))[0][0])  # row 0, block 0
    tb[at] = 0xFF
    _gemm(hm, qa, ta, qb, tb, m, n, k, d)
    got = d.cpu().numpy()
    assert np.isnan(got[1]).all() and np.isnan(got[:, 0]).all()
    b2 = b.copy()
    b2[2, :32] = 0
    ref, bound = OO.product(a, sa, b2, sb)
    keep = np.ones((m, n), bool)
    keep[1], keep[:, 0] = False, False
    assert np.isfinite(got[keep]).all()
    assert (np.abs(got - ref)[keep] <= ((k / 32 + 33) * 2 * U * bound + 1e-37)[keep]).all()


def test_product_extreme_scales(hm, dev):
    """Scales at both ends of UE8M0 whose product stays in fp32."""
    m, n, k = 20, 33, 64
    rng = np.random.default_rng(2)
    a, sa, qa, ta = _operand(dev, rng, m, k, 32)
    b, sb, qb, tb = _operand(dev, rng, n, k, 32)
    sa2, sb2 = np.full_like(sa, 127 + 100), np.full_like(sb, 127 - 110)
    ta = torch.from_numpy(OX.scale_tile_128x4(sa2)).to(dev)
    tb = torch.from_numpy(OX.scale_tile_128x4(sb2)).to(dev)
    d = torch.zeros(m, n, device=dev)
    _gemm(hm, qa, ta, qb, tb, m, n, k, d)
    ref, bound = OO.product(a, sa2, b, sb2)
    _check_product(d, ref, bound, k, False)


def test_product_past_32_bit_offsets(hm, dev):
    """D's rows 2^31 elements apart: byte offsets beyond 32 bits, element offsets beyond 2^31."""
    rng = np.random.default_rng(11)
    m, n, k, ldd = 3, 70, 64, 2 ** 31 + 2
    a, sa, qa, ta = _operand(dev, rng, m, k, 32)
    b, sb, qb, tb = _operand(dev, rng, n, k, 32)
    flat = torch.zeros((m - 1) * ldd + n, dtype=torch.bfloat16, device=dev)
    hm.mxfp8_gemm(qa.data_ptr(), k, ta.data_ptr(), qb.data_ptr(), k, tb.data_ptr(), m, n, k, flat.data_ptr(), ldd,
                  hm.HM_BF16)
    d = torch.stack([flat[i * ldd:i * ldd + n] for i in range(m)])
    ref, bound = OO.product(a, sa, b, sb)
    _check_product(d, ref, bound, k, True)
    assert int(torch.count_nonzero(flat)) == int(torch.count_nonzero(d))


def test_product_on_another_stream(hm, dev):
    rng = np.random.default_rng(12)
    m, n, k = 150, 256, 512
    a, sa, qa, ta = _operand(dev, rng, m, k, 32)
    b, sb, qb, tb = _operand(dev, rng, n, k, 32)
    d = torch.zeros(m, n, device=dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _gemm(hm, qa, ta, qb, tb, m, n, k, d, stream=st.cuda_stream)
    st.synchronize()
    _check_product(d, *OO.product(a, sa, b, sb), k, False)


# ---- quantization --------------------------------------------------------------
QUANT = [
    # rows, cols, dtype, rowwise, transposed, row factor, column factor, block, ldx - cols
    (1, 1, "f32", True, True, False, False, 32, 0),
    (1, 5120, "bf16", True, False, False, False, 32, 0),
    (5, 33, "bf16", True, True, True, True, 32, 3),
    (32, 128, "f32", True, True, False, True, 128, 0),
    (97, 96, "bf16", False, True, True, False, 128, 8),
    (131, 1408, "bf16", True, True, True, True, 32, 0),
    (128, 260, "f32", False, True, False, False, 32, 1),
    (200, 300, "bf16", True, True, False, False, 128, 4),
    (300, 129, "f32", True, False, True, True, 128, 0),
]


def _poison(dev, *shape):
    return torch.full(shape, 0xEE, dtype=torch.uint8, device=dev)


@pytest.mark.parametrize("rows,cols,dtype,rowwise,transposed,rf,cf,block,pad", QUANT)
def test_quantize(hm, dev, rows, cols, dtype, rowwise, transposed, rf, cf, block, pad):
    rng = np.random.default_rng(rows * 5 + cols)
    dt, code = _dt(hm, dtype)
    x = torch.full((rows, cols + pad), float("nan"), dtype=dt, device=dev)
    x[:, :cols] = torch.from_numpy(_spread(rng, rows, cols)).to(dev).to(dt)
    row = torch.from_numpy(rng.uniform(0.3, 3.0, rows).astype(np.float32)).to(dev) if rf else None
    col = torch.from_numpy(rng.uniform(-2.0, 2.0, cols).astype(np.float32)).to(dev) if cf else None
    c32, r32 = _up(cols, 32), _up(rows, 32)
    q, s = _poison(dev, rows, c32 + 16), _poison(dev, hm.mxfp8_tiled_scale_bytes(rows, c32))
    qt, st = _poison(dev, cols, r32 + 32), _poison(dev, hm.mxfp8_tiled_scale_bytes(cols, r32))
    ptr = lambda t, on=True: t.data_ptr() if on and t is not None else 0  # noqa: E731
    hm.mxfp8_quantize(ptr(x), code, rows, cols, cols + pad, ptr(row), ptr(col), block, ptr(q, rowwise),
                      c32 + 16 if rowwise else 0, ptr(s, rowwise), ptr(qt, transposed), r32 + 32 if transposed else 0,
                      ptr(st, transposed))
    torch.cuda.synchronize()
    y = x[:, :cols].float().cpu().numpy()
    if rf:
        y = y * row.cpu().numpy()[:, None]
    if cf:
        y = y * col.cpu().numpy()[None, :]
    for on, codes, scales, src, k32 in ((rowwise, q, s, y, c32), (transposed, qt, st, y.T, r32)):
        if not on:
            assert (codes == 0xEE).all() and (scales == 0xEE).all()
            continue
        oq, osf = OO.quantize(np.ascontiguousarray(src), block)
        assert np.array_equal(codes[:, :k32].cpu().numpy(), oq)
        assert (codes[:, k32:] == 0xEE).all()
        assert np.array_equal(scales.cpu().numpy(), OX.scale_tile_128x4(osf))


def test_quantize_padding_is_positive_zero(hm, dev):
    """Negative factors leave no negative zeros in the padding of either output."""
    rng = np.random.default_rng(77)
    rows, cols = 41, 45
    x = torch.from_numpy(_spread(rng, rows, cols)).to(dev).to(torch.bfloat16)
    row, col = -torch.ones(rows, device=dev), -2 * torch.ones(cols, device=dev)
    for rm, cm in ((row, None), (None, col)):
        q, s = _poison(dev, rows, 64), _poison(dev, 512)
        qt, st = _poison(dev, cols, 64), _poison(dev, 512)
        hm.mxfp8_quantize(x.data_ptr(), hm.HM_BF16, rows, cols, cols, rm.data_ptr() if rm is not None else 0,
                          cm.data_ptr() if cm is not None else 0, 32, q.data_ptr(), 64, s.data_ptr(), qt.data_ptr(), 64,
                          st.data_ptr())
        y = x.float().cpu().numpy() * (-1 if cm is None else -2)
        oq, _ = OO.quantize(y)
        oqt, _ = OO.quantize(np.ascontiguousarray(y.T))
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(qt.cpu().numpy(), oqt)


def test_quantize_nan_inf_and_zeros(hm, dev):
    x = torch.zeros(64, 64, device=dev)
    x[0, 0], x[1, 1], x[2, 2] = float("nan"), float("inf"), -float("inf")
    x[0, 1], x[40, 40] = 1.0, 2.0 ** -140
    q, s = _poison(dev, 64, 64), _poison(dev, 512)
    qt, st = _poison(dev, 64, 64), _poison(dev, 512)
    hm.mxfp8_quantize(x.data_ptr(), hm.HM_F32, 64, 64, 64, 0, 0, 32, q.data_ptr(), 64, s.data_ptr(), qt.data_ptr(), 64,
                      st.data_ptr())
    q, qt = q.cpu().numpy(), qt.cpu().numpy()
    assert q[0, 0] & 0x7F == 0x7F and qt[0, 0] & 0x7F == 0x7F          # NaN stays NaN
    assert q[0, 1] == 0x78                                              # 1 = 256 * 2^-8 beside it
    assert q[1, 1] == 0x7E and q[2, 2] == 0xFE and qt[1, 1] == 0x7E    # +-448
    assert (q[3:40] == 0).all() and q[40, 40] == 0                     # 2^-140 2^127 is below half the smallest code
    sf = s.cpu().numpy()
    assert sf[3 * 16] == 0                                             # a zero block: 2^-127


def test_quantize_past_32_bit_offsets(hm, dev):
    rows, cols, ldx = 3, 40, 2 ** 31 + 6
    rng = np.random.default_rng(21)
    flat = torch.zeros((rows - 1) * ldx + cols, dtype=torch.bfloat16, device=dev)
    x = torch.from_numpy(_spread(rng, rows, cols)).to(torch.bfloat16)
    for r in range(rows):
        flat[r * ldx:r * ldx + cols] = x[r].to(dev)
    q, s = _poison(dev, rows, 64), _poison(dev, 512)
    hm.mxfp8_quantize(flat.data_ptr(), hm.HM_BF16, rows, cols, ldx, 0, 0, 32, q.data_ptr(), 64, s.data_ptr(), 0, 0, 0)
    oq, osf = OO.quantize(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), OX.scale_tile_128x4(osf))


# ---- RMS norm -------------------------------------------------------------------
NORM = [
    # rows, d, dtype, residual, block, ldx - d, ldh - d
    (1, 32, "f32", True, 32, 0, 0),
    (1, 5120, "bf16", True, 32, 0, 0),
    (3, 96, "bf16", False, 128, 8, 0),
    (130, 256, "bf16", True, 128, 0, 16),
    (33, 2048, "f32", True, 32, 8, 8),
    (7, 4128, "bf16", True, 32, 0, 0),
    (5, 8224, "f32", True, 128, 0, 0),
    (2, 16384, "bf16", True, 32, 0, 8),
    (2, 16384, "f32", True, 32, 0, 0),
]


def _row_views(dev, rng, rows, d, ld, dt, std=1.0):
    t = torch.full((rows, ld), float("nan"), dtype=dt, device=dev)
    t[:, :d] = torch.from_numpy((rng.standard_normal((rows, d)) * std).astype(np.float32)).to(dev).to(dt)
    return t


@pytest.mark.parametrize("rows,d,dtype,res,block,px,ph", NORM)
@pytest.mark.parametrize("in_place", [False, True])
def test_rmsnorm(hm, dev, rows, d, dtype, res, block, px, ph, in_place):
    rng = np.random.default_rng(rows * 3 + d)
    dt, code = _dt(hm, dtype)
    x = _row_views(dev, rng, rows, d, d + px, dt)
    r = _row_views(dev, rng, rows, d, d + ph, dt, 3.0) if res else None
    gamma = torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(dev)
    want = x[:, :d].float() + (r[:, :d].float() if res else 0.0)
    want = want.to(dt)
    h = r if in_place and res else torch.full((rows, d + ph), 9.0, dtype=dt, device=dev)
    rstd = torch.zeros(rows, device=dev)
    q, s = _poison(dev, rows, d), _poison(dev, hm.mxfp8_tiled_scale_bytes(rows, d))
    # without a residual h may be left out
    h_ptr = 0 if in_place and not res else h.data_ptr()
    hm.rmsnorm_mxfp8(x.data_ptr(), d + px, r.data_ptr() if res else 0, h_ptr, d + ph, code, rows, d, gamma.data_ptr(),
                     1e-5, block, rstd.data_ptr(), q.data_ptr(), s.data_ptr())
    torch.cuda.synchronize()
    if h_ptr:
        assert torch.equal(h[:, :d], want)
        if not (in_place and res):
            assert (h[:, d:] == 9.0).all()
    ref, _ = OO.rms_norm(_np64(want), _np64(gamma), float(np.float32(1e-5)))
    got = _np64(rstd)
    assert (np.abs(got - ref) <= 32 * U * ref).all()
    y = want.float().cpu().numpy() * rstd.cpu().numpy()[:, None] * gamma.cpu().numpy()
    oq, osf = OO.quantize(y, block)
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(s.cpu().numpy(), OX.scale_tile_128x4(osf))


def test_rmsnorm_zero_row_and_large_values(hm, dev):
    d = 64
    x = torch.zeros(3, d, device=dev)
    x[1] = 1e15
    x[2, 0] = float("nan")
    gamma, rstd = torch.ones(d, device=dev), torch.zeros(3, device=dev)
    q, s = _poison(dev, 3, d), _poison(dev, 512)
    hm.rmsnorm_mxfp8(x.data_ptr(), d, 0, 0, 0, hm.HM_F32, 3, d, gamma.data_ptr(), 1e-5, 32, rstd.data_ptr(),
                     q.data_ptr(), s.data_ptr())
    q, rstd = q.cpu().numpy(), rstd.cpu().numpy()
    assert (q[0] == 0).all() and abs(rstd[0] - 1e-5 ** -0.5) < 1e-4
    assert (np.abs(rstd[1] * 1e15 - 1) < 1e-6) and (q[1] == 0x78).all()   # y = 1 = 256 * 2^-8
    assert np.isnan(rstd[2]) and ((q[2] & 0x7F) == 0x7F).all()


NORM_GRAD = [
    # rows, d, dtype, residual's gradient, lddy - d, ldh - d
    (1, 32, "f32", True, 0, 0),
    (1, 5120, "bf16", True, 0, 0),
    (33, 2048, "f32", True, 8, 16),
    (700, 1408, "bf16", False, 0, 0),
    (1300, 96, "f32", True, 0, 0),
    (9, 8224, "bf16", True, 8, 0),
    (5, 16384, "f32", True, 0, 0),
    (400, 16384, "bf16", True, 0, 0),
]


@pytest.mark.parametrize("rows,d,dtype,res,py,ph", NORM_GRAD)
@pytest.mark.parametrize("alias", [None, "dy", "dres", "h"])
def test_rmsnorm_gradient(hm, dev, rows, d, dtype, res, py, ph, alias):
    if (alias == "dres" and not res) or (alias == "dy" and py != ph):
        pytest.skip("no such alias in this case")
    rng = np.random.default_rng(rows + d)
    dt, code = _dt(hm, dtype)
    dy = _row_views(dev, rng, rows, d, d + py, dt, 0.5)
    dres = _row_views(dev, rng, rows, d, d + ph, dt, 0.5) if res else None
    h = _row_views(dev, rng, rows, d, d + ph, dt, 2.0)
    gamma = torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(dev)
    rstd = torch.rsqrt(h[:, :d].float().square().mean(dim=1) + 1e-5)
    dx = {None: torch.full((rows, d + ph), 9.0, dtype=dt, device=dev), "dy": dy, "dres": dres, "h": h}[alias]
    args = [_np64(t) for t in (dy[:, :d], h[:, :d], gamma, rstd)]
    dres64 = _np64(dres[:, :d]) if res else None
    o_dx, o_dg = OO.rms_norm_grad(*args, dres64)
    acc = alias is not None
    dg = torch.full((d,), 2.0, device=dev)
    ws = torch.empty(hm.rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device=dev)
    hm.rmsnorm_backward(dy.data_ptr(), d + py, dres.data_ptr() if res else 0, h.data_ptr(), dx.data_ptr(), d + ph, code,
                        rows, d, gamma.data_ptr(), rstd.data_ptr(), dg.data_ptr(), acc, ws.data_ptr(), ws.numel())
    torch.cuda.synchronize()
    y64, h64, g64, r64 = args
    xh, t = h64 * r64[:, None], y64 * g64
    size = r64[:, None] * (np.abs(t) + np.abs(xh) * np.mean(np.abs(t * xh), axis=1, keepdims=True))
    tol = 64 * U * (size + (np.abs(dres64) if res else 0.0))
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(o_dx)
    assert (np.abs(_np64(dx[:, :d]) - o_dx) <= tol + 1e-37).all()
    if alias is None:
        assert (dx[:, d:] == 9.0).all()
    want = o_dg + (2.0 if acc else 0.0)
    dg_tol = (rows + 64) * U * np.abs(y64 * xh).sum(axis=0) + 2 * U * np.abs(want)
    assert (np.abs(_np64(dg) - want) <= dg_tol).all()


def test_rmsnorm_gradient_without_rows(hm, dev):
    dg = torch.full((64,), 2.0, device=dev)
    hm.rmsnorm_backward(0, 0, 0, 0, 0, 0, hm.HM_F32, 0, 64, 0, 0, dg.data_ptr(), True, 0, 0)
    assert (dg == 2.0).all()
    hm.rmsnorm_backward(0, 0, 0, 0, 0, 0, hm.HM_F32, 0, 64, 0, 0, dg.data_ptr(), False, 0, 0)
    assert (dg == 0.0).all()


def test_rmsnorm_gradient_matches_differences_of_the_forward_kernel(hm, dev):
    """Central differences of sum(dy y), y from the kernel's own h and rstd (the codes are the
    identity for the gradient).  fp32 rstd has 2^-20 relative noise, y about 1: with a step
    of 0.05 the loss difference carries 64 * 2^-20 / 0.1 = 6e-4, the third-derivative
    term about 0.05^2 / 6 * 1 = 4e-4 of a gradient of order one: 3e-3."""
    rng = np.random.default_rng(31)
    d, eps = 64, 1e-5
    h = torch.from_numpy(rng.standard_normal((1, d)).astype(np.float32)).to(dev)
    dy = torch.from_numpy(rng.standard_normal((1, d)).astype(np.float32)).to(dev)
    gamma = torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(dev)
    rstd = torch.zeros(1, device=dev)
    q, s = _poison(dev, 1, d), _poison(dev, 512)

    def forward(x):
        hm.rmsnorm_mxfp8(x.data_ptr(), d, 0, 0, 0, hm.HM_F32, 1, d, gamma.data_ptr(), eps, 32, rstd.data_ptr(),
                         q.data_ptr(), s.data_ptr())
        return float((_np64(x) * _np64(rstd)[:, None] * _np64(gamma) * _np64(dy)).sum())

    forward(h)
    dx, dg = torch.zeros(1, d, device=dev), torch.zeros(d, device=dev)
    ws = torch.empty(hm.rmsnorm_backward_workspace(1, d), dtype=torch.uint8, device=dev)
    hm.rmsnorm_backward(dy.data_ptr(), d, 0, h.data_ptr(), dx.data_ptr(), d, hm.HM_F32, 1, d, gamma.data_ptr(),
                        rstd.data_ptr(), dg.data_ptr(), False, ws.data_ptr(), ws.numel())
    for c in (0, 13, 63):
        e = torch.zeros_like(h)
        e[0, c] = 0.05
        up, down = h + e, h - e
        step = float(up[0, c].double() - down[0, c].double())
        assert abs((forward(up) - forward(down)) / step - float(dx[0, c])) < 3e-3


# ---- clipping -------------------------------------------------------------------
def _clip(hm, dev, grads, max_norm, place, eps=1e-6):
    """Runs the call on views at odd offsets of one allocation; returns (outputs, norm, coef)."""
    outs, items = [], []
    for i, g in enumerate(grads):
        code = hm.HM_F32 if g.dtype == torch.float32 else hm.HM_BF16
        lead = i % 5
        src = torch.full((g.numel() + lead + 3,), 3.0, dtype=g.dtype, device=dev)
        src[lead:lead + g.numel()] = g.to(dev)
        dst = src if place == "in" else torch.full_like(src, 3.0)
        shift = lead if place != "odd" else (lead + 1) % 4   # dst aligned differently from src
        outs.append((src, dst, lead, shift, g.numel()))
        items.append((src.data_ptr() + lead * g.element_size(),
                      0 if place == "none" else dst.data_ptr() + shift * g.element_size(), g.numel(), code))
    lst = hm.grad_list(items)
    ws = torch.empty(hm.grad_norm_clip_workspace(lst) + 16, dtype=torch.uint8, device=dev)
    stats = torch.zeros(2, device=dev)
    hm.grad_norm_clip(lst, max_norm, eps, stats.data_ptr(), ws.data_ptr(), ws.numel())
    torch.cuda.synchronize()
    norm, coef = stats.cpu().numpy()
    return outs, norm, coef


def _same_bits(a, b):
    v = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.view(v), b.view(v))


CLIP = {
    "one": [("f32", 1)],
    "small": [("f32", 7), ("bf16", 9), ("f32", 0), ("bf16", 1), ("f32", 40000), ("bf16", 32769)],
    "many": [("f32" if i % 3 else "bf16", 100 + 37 * i) for i in range(600)],
    "chunks": [("f32", 16384 * 3 + 5), ("bf16", 32768 * 5 + 11), ("f32", 700001)],
}


@pytest.mark.parametrize("which", list(CLIP))
@pytest.mark.parametrize("place", ["new", "in", "odd", "none"])
@pytest.mark.parametrize("factor", [0.3, 3.0])
def test_clip(hm, dev, which, place, factor):
    rng = np.random.default_rng(len(which))
    grads = [torch.from_numpy(rng.standard_normal(n).astype(np.float32) * 1e-3)
             .to(torch.float32 if t == "f32" else torch.bfloat16) for t, n in CLIP[which]]
    ref, _ = OO.clip([_np64(g) for g in grads], 1.0, 1e-6)
    outs, norm, coef = _clip(hm, dev, grads, float(ref * factor), place)
    assert abs(norm - ref) <= 128 * U * ref
    want = np.float32(min(1.0, float(np.float32(ref * factor)) / (ref + 1e-6)))
    assert abs(coef - want) <= 130 * U
    assert (coef == 1.0) == (factor > 1)
    for g, (src, dst, lead, shift, n) in zip(grads, outs):
        x = g.to(dev)
        y = x if place == "none" else (x.float() * torch.tensor(coef, device=dev)).to(x.dtype)
        if place == "none":
            assert (dst == 3.0).all() and torch.equal(src[lead:lead + n], x)
            continue
        assert _same_bits(dst[shift:shift + n], y)
        assert (dst[:shift] == 3.0).all() and (dst[shift + n:] == 3.0).all()


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-38])
def test_clip_where_squares_leave_fp32(hm, dev, scale):
    rng = np.random.default_rng(6)
    grads = [torch.from_numpy((rng.standard_normal(5000) * scale).astype(np.float32)),
             torch.from_numpy((rng.standard_normal(3000) * scale).astype(np.float32)).to(torch.bfloat16)]
    ref, _ = OO.clip([_np64(g) for g in grads], 1.0, 0.0)
    outs, norm, coef = _clip(hm, dev, grads, float(ref) * 0.5, "new", 0.0)
    assert abs(float(norm) - ref) <= 128 * U * ref
    assert abs(float(coef) - 0.5) <= 130 * U


def test_clip_nan_inf_and_zeros(hm, dev):
    z = [torch.zeros(1000), torch.zeros(77, dtype=torch.bfloat16)]
    outs, norm, coef = _clip(hm, dev, z, 1.0, "new")
    assert norm == 0.0 and coef == 1.0
    outs, norm, coef = _clip(hm, dev, z, 1.0, "new", 0.0)
    assert norm == 0.0 and coef == 1.0
    g = torch.ones(1000)
    g[3] = float("inf")
    outs, norm, coef = _clip(hm, dev, [g], 1.0, "new")
    got = outs[0][1][outs[0][3]:outs[0][3] + 1000]
    assert np.isinf(norm) and coef == 0.0 and torch.isnan(got[3]) and (got[4:] == 0).all()
    g[3] = float("nan")
    outs, norm, coef = _clip(hm, dev, [g, torch.ones(5)], 1.0, "new")
    assert np.isnan(norm) and np.isnan(coef) and torch.isnan(outs[1][1][outs[1][3]:outs[1][3] + 5]).all()
    _, norm, coef = _clip(hm, dev, [torch.ones(64)], float("inf"), "in")
    assert norm == 8.0 and coef == 1.0
    stats = torch.full((2,), 5.0, device=dev)
    hm.grad_norm_clip(hm.grad_list([]), 1.0, 1e-6, stats.data_ptr(), 0, 0)
    assert stats.tolist() == [0.0, 1.0]


def test_operators_in_a_graph(hm, dev):
    """The calls allocate nothing and launch only kernels: a graph replay gives the same bits."""
    rng = np.random.default_rng(41)
    rows, d, n = 70, 256, 384
    x = _row_views(dev, rng, rows, d, d, torch.bfloat16)
    gamma, rstd = torch.ones(d, device=dev), torch.zeros(rows, device=dev)
    q, s = _poison(dev, rows, d), _poison(dev, hm.mxfp8_tiled_scale_bytes(rows, d))
    _, _, qw, tw = _operand(dev, rng, n, d, 32)
    out = torch.zeros(rows, n, device=dev)
    stats = torch.zeros(2, device=dev)
    lst = hm.grad_list([(out.data_ptr(), out.data_ptr(), out.numel(), hm.HM_F32)])
    ws = torch.empty(hm.grad_norm_clip_workspace(lst), dtype=torch.uint8, device=dev)

    def step():
        st = torch.cuda.current_stream().cuda_stream
        hm.rmsnorm_mxfp8(x.data_ptr(), d, 0, 0, 0, hm.HM_BF16, rows, d, gamma.data_ptr(), 1e-5, 32, rstd.data_ptr(),
                         q.data_ptr(), s.data_ptr(), st)
        _gemm(hm, q, s, qw, tw, rows, n, d, out, stream=st)
        hm.grad_norm_clip(lst, 1e-3, 1e-6, stats.data_ptr(), ws.data_ptr(), ws.numel(), st)

    step()
    torch.cuda.synchronize()
    want, want_stats = out.clone(), stats.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x2 = x.clone()
    x.copy_(x2 * 2)
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want) or torch.equal(stats, want_stats)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(stats, want_stats)
    assert hm.hm_device_error() == 0


@pytest.mark.parametrize("m,n,k,out", [
    (1024, 6400, 2208, "f32"),    # 256 x 192 tiles, K summed in two chunks, last one short
    (2304, 3264, 1056, "bf16"),   # 256 x 256 tiles past the last column
    (2000, 3201, 160, "f32"),     # odd pitch: the swapped roles
])
def test_product_tile_widths(hm, dev, m, n, k, out):
    """Every tile width of the persistent kernel, against float64 on the GPU (too large for the host)."""
    g = torch.Generator(device=dev)
    g.manual_seed(m + n)
    ops = []
    for rows in (m, n):
        codes = torch.randint(0, 256, (rows, k), generator=g, device=dev, dtype=torch.uint8)
        codes[codes & 0x7F == 0x7F] = 0x10
        sf = torch.randint(120, 131, (rows, k // 32), generator=g, device=dev, dtype=torch.uint8)
        tiled = torch.from_numpy(OX.scale_tile_128x4(sf.cpu().numpy())).to(dev)
        val = codes.view(torch.float8_e4m3fn).double().view(rows, -1, 32) * torch.exp2(sf.double() - 127)[:, :, None]
        ops.append((codes, tiled, val.view(rows, k)))
    (qa, ta, va), (qb, tb, vb) = ops
    d = torch.zeros(m, n, dtype=_dt(hm, out)[0], device=dev)
    _gemm(hm, qa, ta, qb, tb, m, n, k, d)
    ref, bound = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = (k / 32 + 33) * 2 * U * bound
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert bool(((d.double() - ref).abs() <= tol).all())
    assert hm.hm_device_error() == 0


@pytest.mark.parametrize("m,n,k", [(1, 300, 12288), (40, 200, 24576), (300, 260, 8192)])
def test_product_long_fp32_sums(hm, dev, m, n, k):
    """fp32 D over a long K, operands of one sign (every truncation of the accumulator goes the
    same way): no chain of tensor-core additions is longer than 2560, so the error stays
    within (2560 / 32 + 33) 2u of the sum plus one rounding per part."""
    g = torch.Generator(device=dev)
    g.manual_seed(k)
    ops = []
    for rows in (m, n):
        codes = torch.randint(0x30, 0x40, (rows, k), generator=g, device=dev, dtype=torch.uint8)
        sf = torch.full((rows, k // 32), 127, device=dev, dtype=torch.uint8)
        tiled = torch.from_numpy(OX.scale_tile_128x4(sf.cpu().numpy())).to(dev)
        ops.append((codes, tiled, codes.view(torch.float8_e4m3fn).double()))
    (qa, ta, va), (qb, tb, vb) = ops
    d = torch.zeros(m, n, device=dev)
    _gemm(hm, qa, ta, qb, tb, m, n, k, d)
    ref = va @ vb.t()
    assert bool(((d.double() - ref).abs() <= ((2560 / 32 + 33) * 2 + k / 2048 + 8) * U * ref).all())


@pytest.mark.parametrize("count,n", [(16, 3000), (17, 3000), (1, 2 ** 18), (1, 2 ** 18 + 9), (1, 2 ** 18 + 4096), (3, 400000)])
@pytest.mark.parametrize("place", ["new", "in", "odd"])
def test_clip_around_the_one_launch_form(hm, dev, count, n, place):
    """Tensor counts and sizes on both sides of where one launch does it all: the same values."""
    rng = np.random.default_rng(n + count)
    grads = [torch.from_numpy(rng.standard_normal(n - 3 * i).astype(np.float32)) for i in range(count)]
    ref, _ = OO.clip([_np64(g) for g in grads], 1.0, 1e-6)
    before = hm.hm_kernel_launches()
    outs, norm, coef = _clip(hm, dev, grads, float(ref) * 0.5, place)
    few = count <= 16 and 4 * n * count <= 2 ** 20 + 16   # a tail of less than a vector takes no chunk
    assert hm.hm_kernel_launches() - before == (1 if few else 2) or n == 2 ** 18 + 9
    assert abs(norm - ref) <= 128 * U * ref and abs(coef - 0.5) <= 130 * U
    for g, (src, dst, lead, shift, k) in zip(grads, outs):
        assert _same_bits(dst[shift:shift + k], g.to(dev) * torch.tensor(coef, device=dev))


@pytest.mark.parametrize("which", ["pair", "sums", "split", "one", "norm_grad"])
def test_injected_wait_timeout_is_reported_and_recovered(hm, dev, which):
    """An accumulator that is never marked ready (pair: CTA pairs, sums: with K in chunks, split:
    a cluster per tile, one: a CTA per tile), or rows that never arrive: the bounded waits
    give up, record HM_ERR_TIMEOUT and return; the next call is right."""
    import os
    rng = np.random.default_rng(5)
    if which == "norm_grad":
        rows, d = 40, 2048
        dy, h = (torch.randn(rows, d, device=dev) for _ in range(2))
        gamma, rstd = torch.ones(d, device=dev), torch.ones(rows, device=dev)
        dx, dg = torch.zeros(rows, d, device=dev), torch.zeros(d, device=dev)
        ws = torch.empty(hm.rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device=dev)
        ref = OO.rms_norm_grad(_np64(dy), _np64(h), _np64(gamma), _np64(rstd))[0]

        def call():
            hm.rmsnorm_backward(dy.data_ptr(), d, 0, h.data_ptr(), dx.data_ptr(), d, hm.HM_F32, rows, d, gamma.data_ptr(),
                                rstd.data_ptr(), dg.data_ptr(), False, ws.data_ptr(), ws.numel())

        def right():
            return np.allclose(_np64(dx), ref, rtol=1e-5, atol=1e-4)
    else:
        m, n, k, t = {"pair": (2304, 3264, 1056, "bf16"), "sums": (1024, 6400, 2208, "f32"), "split": (5, 256, 2048, "f32"),
                      "one": (5, 256, 64, "f32")}[which]
        a = torch.full((m, k), 0x38, dtype=torch.uint8, device=dev)   # 1.0
        b = torch.full((n, k), 0x38, dtype=torch.uint8, device=dev)
        sa, sb = (torch.full((hm.mxfp8_tiled_scale_bytes(r, k),), 127, dtype=torch.uint8, device=dev) for r in (m, n))
        d = torch.zeros(m, n, dtype=_dt(hm, t)[0], device=dev)

        def call():
            _gemm(hm, a, sa, b, sb, m, n, k, d)

        def right():
            return bool((d == k).all())
    assert hm.hm_device_error() == 0
    os.environ["HM_INJECT_MX_WAIT_TIMEOUT"] = "1"
    try:
        call()
        torch.cuda.synchronize()                  # returns: the waits are bounded
    finally:
        del os.environ["HM_INJECT_MX_WAIT_TIMEOUT"]
    assert hm.hm_device_error() == hm.HM_ERR_TIMEOUT
    assert hm.hm_device_error() == 0              # read-and-clear
    call()
    torch.cuda.synchronize()
    assert hm.hm_device_error() == 0 and right()


def test_clip_infinite_max_norm(hm, dev):
    """An infinite max_norm never clips, whatever the norm; a NaN still shows."""
    g = torch.ones(100)
    g[7] = float("inf")
    outs, norm, coef = _clip(hm, dev, [g], float("inf"), "new")
    assert np.isinf(norm) and coef == 1.0 and torch.equal(outs[0][1][outs[0][3]:outs[0][3] + 100].cpu(), g)
    g[8] = float("nan")
    _, norm, coef = _clip(hm, dev, [g], float("inf"), "new")
    assert np.isnan(norm) and np.isnan(coef)


@pytest.mark.parametrize("factors", [False, True])
def test_quantize_bf16_nan_inf_and_zeros(hm, dev, factors):
    """The same special values in bf16, with and without factors."""
    x = torch.zeros(64, 64, device=dev, dtype=torch.bfloat16)
    x[0, 0], x[1, 1], x[2, 2] = float("nan"), float("inf"), -float("inf")
    x[0, 1], x[3, 3] = 1.0, 2.0 ** -133    # the smallest subnormal: 2^-133 2^127 = 2^-6
    one = torch.ones(64, device=dev)
    q, s = _poison(dev, 64, 64), _poison(dev, 512)
    qt, st = _poison(dev, 64, 64), _poison(dev, 512)
    f = one.data_ptr() if factors else 0
    hm.mxfp8_quantize(x.data_ptr(), hm.HM_BF16, 64, 64, 64, f, f, 32, q.data_ptr(), 64, s.data_ptr(), qt.data_ptr(), 64,
                      st.data_ptr())
    q, qt = q.cpu().numpy(), qt.cpu().numpy()
    assert q[0, 0] & 0x7F == 0x7F and qt[0, 0] & 0x7F == 0x7F          # NaN stays NaN
    assert q[0, 1] == 0x78                                              # 1 = 256 * 2^-8
    assert q[1, 1] == 0x7E and q[2, 2] == 0xFE and qt[1, 1] == 0x7E    # +-448
    assert q[3, 3] == 0x08 and qt[3, 3] == 0x08                        # 2^-6, the smallest normal code
    assert (q[4:] == 0).all() and (qt[4:] == 0).all()
    assert s.cpu().numpy()[4 * 16] == 0
