"""Every kernel form that a product with an epilogue takes, with aligned rows and odd
ones, against the product in 64 bits on the GPU.

Tolerances: z as in the products' own forms, (K/32 + 33) 2u sum |a b| (u = 2^-24, one
rounding more with a bias); SiLU's slope is below 1.1 and its evaluation off by less
than 16u |x| in value and 32u (1 + |x|) in slope (x s(x): exp2 within 4u after an
argument off by 3u |x|, the quotient within 2u, |x| s (1 - s) <= 0.23); a bf16
output adds half a step, 2^-8 of it.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _up(x, k):
    return -(-x // k) * k


def _operand(g, dev, rows, k):
    """Codes (no NaN), tiled scales with NaN in their padding, and the values in 64 bits."""
    codes = torch.randint(0, 256, (rows, k), generator=g, device=dev, dtype=torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0x10
    sf = torch.randint(114, 118, (rows, k // 32), generator=g, device=dev, dtype=torch.uint8)
    full = torch.full((_up(rows, 128), _up(k // 32, 4)), 0xFF, dtype=torch.uint8, device=dev)
    full[:rows, :k // 32] = sf
    tiled = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    val = codes.view(torch.float8_e4m3fn).double().view(rows, -1, 32) * torch.exp2(sf.double() - 127)[:, :, None]
    return codes, tiled, val.view(rows, k)


FORMS = [
    # m, n, k, D, (tile, parts, sums)
    (2311, 1400, 6432, "bf16", (256, 0, 0)),
    (1030, 6403, 3104, "bf16", (256, 0, 0)),   # several tiles per pair, here and below
    (2311, 4099, 96, "bf16", (192, 0, 0)),
    (4000, 6400, 1056, "f32", (192, 0, 0)),
    (2311, 6403, 1056, "bf16", (128, 0, 0)),
    (2048, 9728, 1920, "f32", (128, 0, 0)),
    (1030, 4099, 3104, "f32", (192, 0, 1)),    # two chunks
    (2311, 1400, 2080, "f32", (128, 0, 1)),
    (617, 9731, 2080, "f32", (128, 0, 1)),
    (5, 300, 24576, "f32", (128, 0, 1)),       # twelve chunks
    (1900, 2560, 160, "bf16", (128, 1, 0)),
    (1541, 1400, 3104, "bf16", (128, 2, 0)),
    (65, 2600, 544, "f32", (128, 5, 0)),
    (600, 700, 96, "bf16", (64, 1, 0)),
    (515, 1030, 4128, "f32", (64, 3, 0)),
    (40, 130, 6432, "bf16", (64, 8, 0)),
    (17, 130, 544, "f32", (32, 5, 0)),
    (17, 130, 64, "bf16", (32, 1, 0)),
    (1, 130, 160, "f32", (16, 2, 0)),
    (1, 130, 64, "bf16", (16, 1, 0)),
]


@pytest.mark.parametrize("m,n,k,out,form", FORMS)
@pytest.mark.parametrize("aligned", [True, False])
def test_epilogue_form(hm, dev, m, n, k, out, form, aligned):
    assert hm.mxfp8_gemm_epilogue_form(m, n, k, hm.HM_F32 if out == "f32" else hm.HM_BF16) == form
    if aligned:
        n = _up(n, 8)  # the same number of tiles
        assert hm.mxfp8_gemm_epilogue_form(m, n, k, hm.HM_F32 if out == "f32" else hm.HM_BF16) == form
    ld = n + (8 if aligned else 3)
    g = torch.Generator(device=dev)
    g.manual_seed(m + n + k)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    qa, ta, va = _operand(g, dev, m, k)
    qb, tb, vb = _operand(g, dev, n, k)
    z, bound = va @ vb.t(), va.abs() @ vb.abs().t()
    std = float(z.std())
    ez = (k / 32 + 33) * 2 * U * bound
    del va, vb, bound
    new = lambda: torch.randn(m, ld, generator=g, device=dev).to(dt)  # noqa: E731
    gate, up, bias = new(), new(), torch.randn(n, generator=g, device=dev) * std
    guard = lambda: torch.full((m + 1, ld), 7.0, dtype=dt, device=dev)  # noqa: E731
    d, out2 = guard(), guard()
    p = lambda t: t.data_ptr()  # noqa: E731

    def call(e):
        hm.mxfp8_gemm_epilogue(p(qa), k, p(ta), p(qb), k, p(tb), m, n, k, p(d), ld, hm.HM_F32 if out == "f32" else hm.HM_BF16, e)

    def near(got, want, tol):
        assert (got[m] == 7).all() and (got[:, n:] == 7).all(), "a row or column past D was written"
        tol = tol + 4 * U * want.abs()
        if out == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        err = (got[:m, :n].double() - want).abs()
        assert bool(torch.isfinite(err).all()) and bool((err <= tol + 1e-30).all()), float((err / (tol + 1e-30)).max())

    zb = z + bias.double()
    s = torch.sigmoid(zb)
    call(hm.hm_epilogue(hm.HM_EPI_FORWARD, hm.HM_ACT_SILU, p(bias), p(gate), ld, 0, 0, p(out2), ld))
    eb = ez + 2 * U * zb.abs()
    near(d, zb * s + gate[:, :n].double(), 1.1 * eb + 16 * U * zb.abs())
    near(out2, zb, eb)
    del zb, s, eb
    x, y = gate[:, :n].double(), up[:, :n].double()
    s = torch.sigmoid(x)
    slope = s + x * s * (1 - s)
    call(hm.hm_epilogue(hm.HM_EPI_GATED_GRADIENT, hm.HM_ACT_SILU, 0, p(gate), ld, p(up), ld, p(out2), ld))
    near(d, z * x * s, (x * s).abs() * ez + z.abs() * 16 * U * x.abs())
    near(out2, z * y * slope, y.abs() * (slope.abs() * ez + z.abs() * 32 * U * (1 + x.abs())))
    assert hm.hm_device_error() == 0
