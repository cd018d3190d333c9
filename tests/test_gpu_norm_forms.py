"""The norm and its gradient where a warp or a CTA takes several rows, and at every
width's kernel form, against float64.  Tolerances (by derivation, u = 2^-24) as in the operators' tests:
rstd 32 u; dx 64 u of its terms' magnitudes, plus 2^-8 |dx| for bf16; dgamma
(rows + 64) u sum |dy xhat|; h, codes and scales bit-exact."""
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


def _rows(dev, g, rows, d, ld, dt, std):
    t = torch.full((rows, ld), float("nan"), dtype=dt, device=dev)
    t[:, :d] = (torch.randn(rows, d, generator=g, device=dev) * std).to(dt)
    return t


GRAD = [
    # rows, d, residual's gradient, lddy - d, ldh - d
    (5001, 256, True, 0, 0),      # a warp per row, at most 4864 at a time: some take a second one
    (20011, 96, True, 8, 8),      # five rows per warp
    (2500, 512, True, 0, 8),      # 2432 rows at a time
    (2500, 992, False, 0, 0),
    (7400, 1024, True, 0, 0),
    (2000, 1056, True, 0, 0),     # a CTA per row from here on, several rows each
    (1500, 4096, True, 8, 0),
    (1000, 5120, False, 0, 0),
    (900, 6656, True, 0, 0),
    (700, 8192, True, 0, 0),
    (900, 8224, False, 0, 0),
]


@pytest.mark.parametrize("rows,d,res,py,ph", GRAD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("alias", [None, "dy", "dres", "h"])
def test_gradient_of_several_rows_each(hm, dev, rows, d, res, py, ph, dtype, alias):
    if (alias == "dres" and not res) or (alias == "dy" and py != ph):
        pytest.skip("no such alias in this case")
    g = torch.Generator(device=dev)
    g.manual_seed(rows + d)
    dt, code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
    dy = _rows(dev, g, rows, d, d + py, dt, 0.5)
    dres = _rows(dev, g, rows, d, d + ph, dt, 0.5) if res else None
    h = _rows(dev, g, rows, d, d + ph, dt, 2.0)
    # rows of different sizes: a neighbour's rstd, or its row, would show
    h[:, :d] *= torch.exp2(torch.arange(rows, device=dev) % 7 - 3.0).to(dt)[:, None]
    gamma = 1 + 0.1 * torch.randn(d, generator=g, device=dev)
    rstd = torch.rsqrt(h[:, :d].float().square().mean(dim=1) + 1e-5)
    y64, h64, g64, r64 = dy[:, :d].double(), h[:, :d].double(), gamma.double(), rstd.double()
    dres64 = dres[:, :d].double() if res else torch.zeros_like(y64)
    xh, t = h64 * r64[:, None], y64 * g64
    want = dres64 + r64[:, None] * (t - xh * (t * xh).mean(dim=1, keepdim=True))
    tol = 64 * U * (dres64.abs() + r64[:, None] * (t.abs() + xh.abs() * (t * xh).abs().mean(dim=1, keepdim=True)))
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * want.abs()
    want_g, tol_g = (y64 * xh).sum(dim=0), (rows + 64) * U * (y64 * xh).abs().sum(dim=0)
    acc = alias == "dy"
    if acc:
        want_g = want_g + 2.0
        tol_g = tol_g + 2 * U * want_g.abs()
    dx = {None: torch.full((rows, d + ph), 9.0, dtype=dt, device=dev), "dy": dy, "dres": dres, "h": h}[alias]
    dg = torch.full((d,), 2.0, device=dev)
    ws = torch.full((hm.rmsnorm_backward_workspace(rows, d),), 0xFF, dtype=torch.uint8, device=dev)
    hm.rmsnorm_backward(dy.data_ptr(), d + py, dres.data_ptr() if res else 0, h.data_ptr(), dx.data_ptr(), d + ph, code,
                        rows, d, gamma.data_ptr(), rstd.data_ptr(), dg.data_ptr(), acc, ws.data_ptr(), ws.numel())
    torch.cuda.synchronize()
    assert hm.hm_device_error() == 0
    assert bool(((dx[:, :d].double() - want).abs() <= tol + 1e-37).all())
    if alias is None:
        assert bool((dx[:, d:] == 9.0).all())
    assert bool(((dg.double() - want_g).abs() <= tol_g + 2 * U * want_g.abs()).all())


@pytest.mark.parametrize("rows,d", [(300, 288), (140, 512), (11, 544), (129, 992), (70, 1024), (9, 1056), (5, 8192)])
@pytest.mark.parametrize("dtype,res,block", [("bf16", True, 32), ("f32", False, 128), ("f32", True, 32), ("bf16", False, 128)])
def test_norm_at_every_width(hm, dev, rows, d, dtype, res, block):
    g = torch.Generator(device=dev)
    g.manual_seed(rows + d)
    dt, code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
    x = _rows(dev, g, rows, d, d + 8, dt, 1.0)
    x[:, :d] *= torch.exp2(torch.arange(rows, device=dev) % 9 - 4.0).to(dt)[:, None]
    r = _rows(dev, g, rows, d, d + 16, dt, 3.0) if res else None
    gamma = 1 + 0.1 * torch.randn(d, generator=g, device=dev)
    h = torch.full((rows, d + 16), 9.0, dtype=dt, device=dev)
    rstd = torch.zeros(rows, device=dev)
    q = torch.full((rows, d), 0xEE, dtype=torch.uint8, device=dev)
    s = torch.full((hm.mxfp8_tiled_scale_bytes(rows, d),), 0xEE, dtype=torch.uint8, device=dev)
    hm.rmsnorm_mxfp8(x.data_ptr(), d + 8, r.data_ptr() if res else 0, h.data_ptr(), d + 16, code, rows, d,
                     gamma.data_ptr(), 1e-5, block, rstd.data_ptr(), q.data_ptr(), s.data_ptr())
    torch.cuda.synchronize()
    want = (x[:, :d].float() + (r[:, :d].float() if res else 0.0)).to(dt)
    assert torch.equal(h[:, :d], want) and bool((h[:, d:] == 9.0).all())
    ref = (want.double().square().mean(dim=1) + float(np.float32(1e-5))) ** -0.5
    assert bool(((rstd.double() - ref).abs() <= 32 * U * ref).all())
    y = want.float().cpu().numpy() * rstd.cpu().numpy()[:, None] * gamma.cpu().numpy()
    oq, osf = OO.quantize(y, block)
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(s.cpu().numpy(), OX.scale_tile_128x4(osf))
