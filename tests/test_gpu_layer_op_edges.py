"""Edges that depend on how many CTAs a GPU gives a call: the heads' positions that just fit in
shared memory beside the angles and those that do not, and the chunked sums of an epilogue.

Tolerances as test_gpu_layer_ops.py derives them (u = 2^-24): heads 24u (|a| + |b|) of a pair
with each at its head's largest, 48u, and half a bf16 step; the product's z off by
(K/32 + 33) 2u sum |a b|, SiLU by 16u |x|, its slope by 32u (1 + |x|).
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


# The forward pass runs a whole number of times the resident CTAs, the more the more rounds of
# all a CTA's slots there are: 256 slots at 16 elements, 64 at 64, so that one wave is left
# with 1024 rows of two single heads each (4 CTAs per SM, 3 in fp32, 2 with narrow vectors).
@pytest.mark.parametrize("extra", [-1, 0, 1])
@pytest.mark.parametrize("dtype,dim,rot,ctas", [("bf16", 16, 16, 4), ("bf16", 32, 16, 4), ("f32", 16, 8, 3), ("bf16", 12, 4, 2)])
def test_forward_positions_that_just_fit(hm, dev, extra, dtype, dim, rot, ctas):
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    rows = 1024 * (ctas * sms // 2) + extra     # half the CTAs for each group: 1024 rows, or one CTA one less or more
    dt, code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
    g = torch.Generator(device=dev)
    g.manual_seed(dim)
    x = torch.randn(rows, 2, dim, generator=g, device=dev).to(dt)
    out = torch.full((rows + 1, 2, dim), 7.0, device=dev, dtype=dt)
    pos = torch.randint(0, 100000, (rows,), generator=g, device=dev)
    turns, _ = hm.rope_turns(rot)
    table = torch.tensor(turns, dtype=torch.int64, device=dev)
    rotation = hm.hm_rotation(table.data_ptr(), pos.data_ptr(), 1.0, rot, hm.HM_ROPE_HALF)
    es = x.element_size()
    at = lambda t, h: (t.data_ptr() + es * h * dim, 2 * dim, dim)  # noqa: E731
    hm.head_norm_rope(hm.head_list([(*at(x, h), *at(out, h), 0, 1) for h in range(2)]), code, rows, dim, 1e-5, rotation)
    f = table.double() * (2 * torch.pi / 2.0 ** 64)
    a = pos.double()[:, None, None] * f
    v = x.double()
    u, w = v[..., :rot // 2], v[..., rot // 2:rot]
    want = torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin(), v[..., rot:]], -1)
    tol = 48 * U * v.abs().amax(-1, keepdim=True)
    # 2 pi in 64 bits times 1e5 positions is off by less than u / 100
    half = 2.0 ** -8 if dtype == "bf16" else U
    assert (out[rows] == 7).all()
    assert bool(((out[:rows].double() - want).abs() <= tol * (1 + half) + half * want.abs()).all())
    assert hm.hm_device_error() == 0


@pytest.mark.parametrize("m,n,k", [(4200, 2600, 4128), (70, 300, 24608)])
@pytest.mark.parametrize("form", ["forward", "gated_gradient"])
@pytest.mark.parametrize("pad", [0, 1])
def test_chunked_sums_with_an_epilogue(hm, dev, m, n, k, form, pad):
    tile, parts, sums = hm.mxfp8_gemm_epilogue_form(m, n, k, hm.HM_F32)
    assert (parts, sums) == (0, 1)
    g = torch.Generator(device=dev)
    g.manual_seed(k)
    code = lambda rows: torch.randint(0, 256, (rows, k), generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    qa, qb = code(m), code(n)
    for q in (qa, qb):
        q[q & 0x7F == 0x7F] = 0x10
    sa = torch.full((hm.mxfp8_tiled_scale_bytes(m, k),), 116, dtype=torch.uint8, device=dev)
    sb = torch.full((hm.mxfp8_tiled_scale_bytes(n, k),), 115, dtype=torch.uint8, device=dev)
    va, vb = (q.view(torch.float8_e4m3fn).double() * 2.0 ** s for q, s in ((qa, -11), (qb, -12)))
    z, ez = va @ vb.t(), (k / 32 + 33) * 2 * U * (va.abs() @ vb.abs().t())
    del va, vb
    ld = n + pad
    new = lambda: torch.randn(m, ld, generator=g, device=dev)  # noqa: E731
    first, second, bias = new(), new(), torch.randn(n, generator=g, device=dev)
    d, out2 = (torch.full((m + 1, ld), 7.0, device=dev) for _ in range(2))
    p = lambda t: t.data_ptr()  # noqa: E731
    e = (hm.hm_epilogue(hm.HM_EPI_FORWARD, hm.HM_ACT_SILU, p(bias), p(first), ld, 0, 0, p(out2), ld) if form == "forward" else
         hm.hm_epilogue(hm.HM_EPI_GATED_GRADIENT, hm.HM_ACT_SILU, 0, p(first), ld, p(second), ld, p(out2), ld))
    hm.mxfp8_gemm_epilogue(p(qa), k, p(sa), p(qb), k, p(sb), m, n, k, p(d), ld, hm.HM_F32, e)

    def near(got, want, tol):
        assert (got[m] == 7).all() and (got[:, n:] == 7).all()
        err = (got[:m, :n].double() - want).abs()
        assert bool((err <= tol + 4 * U * want.abs() + 1e-30).all()), float((err / (tol + 4 * U * want.abs() + 1e-30)).max())

    x, y = first[:, :n].double(), second[:, :n].double()
    if form == "forward":
        zb = z + bias.double()
        eb = ez + 2 * U * zb.abs()
        near(d, zb * torch.sigmoid(zb) + x, 1.1 * eb + 16 * U * zb.abs())
        near(out2, zb, eb)
    else:
        s = torch.sigmoid(x)
        slope = s + x * s * (1 - s)
        near(d, z * x * s, (x * s).abs() * ez + z.abs() * 16 * U * x.abs())
        near(out2, z * y * slope, y.abs() * (slope.abs() * ez + z.abs() * 32 * U * (1 + x.abs())))
    assert hm.hm_device_error() == 0


def test_forms_have_their_kernels(hm, dev):
    """The epilogue's kernels exist for the tiles that the choice can name: fp32 on pairs of at most
    192 rows, sums of chunks in fp32 only."""
    seen = set()
    for m in (1, 17, 40, 100, 300, 777, 2048, 8192, 40000):
        for n in (8, 1408, 4096, 20480):
            for k in (32, 1024, 2048, 2080, 5120, 24576):
                for dtype in (hm.HM_BF16, hm.HM_F32):
                    tile, parts, sums = hm.mxfp8_gemm_epilogue_form(m, n, k, dtype)
                    seen.add((tile, parts > 0, sums))
                    if parts:
                        assert tile in (16, 32, 64, 128) and not sums
                    elif dtype == hm.HM_F32:
                        assert tile in (128, 192)
                    else:
                        assert tile in (128, 192, 256) and not sums
    assert {(256, False, 0), (192, False, 0), (128, False, 1), (192, False, 1), (16, True, 0)} <= seen
