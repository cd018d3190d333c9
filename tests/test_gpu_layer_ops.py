"""The operators of a layer's projections against the float64 oracle, through the C ABI.

Tolerances (by derivation, u = 2^-24; a bf16 output adds half a step, 2^-8 of it):
  epilogue  the product's z is off by e_z = (K/32 + 33) 2u sum |a b| (tests of the
            product), one rounding more with a bias, 2u |z|.  Every activation's slope
            is below 1.13.  Its own evaluation: SiLU and the tanh form are x s(w), s
            the logistic function: w has three roundings, so exp(-w) is off by 3u |w|
            plus expf's and the quotient's 6u; s (1 - s) |w| <= 0.23, so s is off by
            less than 8u and f by 9u |x|; GELU: erfcf's 4 units and its argument's rounding,
            less than 10u |x|.  So 16u |x|.  The slope adds x s (1 - s) w':
            32u (1 + |x| w'), w' <= 1.6 + 0.22 x^2, or 32u (1 + |x|) where w' = 1.
  bias      sums of 32 rows, then 4, the tiles' 32nd parts and 32: (70 + rows / 4096) u sum |x|.
  heads     v = x r gamma: the sum of squares is a chain of at most 16 products and 5
            joins per lane, 21u, half of that in r, 2u for the root, two products: 15u.
            sin and cos: the eighth of a turn's rounding, the function's two units and
            the scale's rounding, 4u of the scale; the pair's products 2u:
            24u scale (|a| + |b|) for a pair (a, b).
  gradient  t as above with 6u; dx: the sums' 30u, three factors of r (13u each) and
            5 products: 96u r (U + |xhat| mean(U |xhat|)), U = |gamma| scale (|da| + |db|);
            dgamma: (N + 64 + 24) u sum T |xhat| over its N rows and heads, T = scale (|da| + |db|).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layers as OL  # noqa: E402
from oracle import mxfp8 as OX  # noqa: E402
from oracle import operators as OO  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FORMS = ("forward", "gated", "gradient", "gated_gradient")


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _code(hm, t):
    return hm.HM_BF16 if t.dtype == torch.bfloat16 else hm.HM_F32


def _operand(dev, rng, rows, k, block):
    codes, sf = OO.quantize((rng.standard_normal((rows, k)) * 0.2).astype(np.float32), block)
    real = OX.scale_tile_128x4(np.ones_like(sf)) == 1
    tiled = np.where(real, OX.scale_tile_128x4(sf), 0xFF).astype(np.uint8)
    return codes, sf, torch.from_numpy(codes).to(dev), torch.from_numpy(tiled).to(dev)


class _Product:
    """Operands, the epilogue's matrices and the call; one row and `pad` columns of guard each."""

    def __init__(self, hm, dev, form, act, m, n, k, out, pad=0, bias=True, first=True, keep=True, block=32, seed=0):
        rng = np.random.default_rng(seed + m * 7 + n * 3 + k)
        self.hm, self.form, self.act, self.m, self.n, self.k, self.pad = hm, form, act, m, n, k, pad
        self.dt = _type(out)
        if k:
            self.a, self.sa, self.qa, self.ta = _operand(dev, rng, m, k, block)
            self.b, self.sb, self.qb, self.tb = _operand(dev, rng, n, k, block)
        grad = form in ("gradient", "gated_gradient")
        new = lambda std: torch.from_numpy(rng.standard_normal((m + 1, n + pad)).astype(np.float32) * np.float32(std)).to(dev).to(self.dt)  # noqa: E731
        self.bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev) if bias and not grad else None
        self.first = new(1.5) if form != "forward" or first else None
        self.second = new(1.0) if form == "gated_gradient" else None
        self.out2 = torch.full((m + 1, n + pad), 7.0, dtype=self.dt, device=dev) if form == "gated_gradient" or (keep and not grad) else None
        self.d = torch.full((m + 1, n + pad), 7.0, dtype=self.dt, device=dev)

    def call(self, stream=0):
        hm, ld = self.hm, self.n + self.pad
        p = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
        e = hm.hm_epilogue(FORMS.index(self.form), OL.ACTS.index(self.act), p(self.bias), p(self.first), ld, p(self.second), ld,
                           p(self.out2), ld)
        ops = (p(self.qa), self.k, p(self.ta), p(self.qb), self.k, p(self.tb)) if self.k else (0, 0, 0, 0, 0, 0)
        hm.mxfp8_gemm_epilogue(*ops, self.m, self.n, self.k, p(self.d), ld, _code(hm, self.d), e, stream)

    def check(self):
        m, n = self.m, self.n
        z, bound = OO.product(self.a, self.sa, self.b, self.sb) if self.k else (np.zeros((m, n)), np.zeros((m, n)))
        ez = (self.k / 32 + 33) * 2 * U * bound
        bias = None if self.bias is None else _np64(self.bias)
        first, second = (None if t is None else _np64(t)[:m, :n] for t in (self.first, self.second))
        d, out2 = OL.epilogue(self.form, self.act, z, bias, first, second)
        if bias is not None:
            z = z + bias
            ez = ez + 2 * U * np.abs(z)
        x = z if self.form == "forward" else first
        f, slope = OL.activate(self.act, x)
        ef = 16 * U * np.abs(x)
        es = 32 * U * (1 + np.abs(x) * (1.6 + 0.22 * x * x if self.act == "gelu_tanh" else 1.0))
        if self.form == "forward":
            tol, tol2 = 1.13 * ez + ef, ez
        elif self.form == "gated":
            tol, tol2 = np.abs(f) * ez + np.abs(z) * ef, ez
        elif self.form == "gradient":
            tol, tol2 = np.abs(slope) * ez + np.abs(z) * es, None
        else:
            tol = np.abs(f) * ez + np.abs(z) * ef
            tol2 = np.abs(second) * (np.abs(slope) * ez + np.abs(z) * es)
        self._near(self.d, d, tol)
        if self.out2 is not None:
            self._near(self.out2, out2, tol2)

    def _near(self, got, want, tol):
        g = _np64(got)
        assert (g[self.m] == 7).all() and (g[:, self.n:] == 7).all(), "a row or column past D was written"
        tol = tol + 4 * U * np.abs(want)
        if self.dt == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        err = np.abs(g[:self.m, :self.n] - want)
        assert np.isfinite(err).all() and (err <= tol + 1e-37).all(), f"worst excess {np.max(err / (tol + 1e-37))}"


# one shape at least for each of the product's kernels: tiles of 16 to 128 rows whole and
# split, pairs of each width, chunked sums (fp32, K > 2048)
SHAPES = [(1, 33, 32), (1, 5120, 1024), (5, 130, 96), (16, 128, 1024), (17, 257, 160), (33, 256, 416), (65, 320, 2080),
          (77, 1408, 2048), (129, 256, 128), (300, 700, 1056), (513, 1030, 640), (3000, 2600, 544)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_epilogue(hm, dev, i, shape, form, out):
    act = OL.ACTS[(i + FORMS.index(form)) % len(OL.ACTS)]
    p = _Product(hm, dev, form, act, *shape, out, pad=(0, 3, -shape[1] % 8)[i % 3], bias=i % 2 == 0, first=i % 3 != 1, keep=i % 4 != 2,
                 block=(32, 128)[i % 2])
    p.call()
    p.check()
    assert hm.hm_device_error() == 0


@pytest.mark.parametrize("form", ["forward", "gated_gradient"])
def test_epilogue_of_chunked_sums(hm, dev, form):
    m, n, k = 400, 2200, 4128
    assert hm.mxfp8_gemm_form(m, n, k, hm.HM_F32)[2] == 1 or m < 1000
    for m in (400, 2100):
        p = _Product(hm, dev, form, "silu", m, n, k, "f32", pad=1)
        p.call()
        p.check()


@pytest.mark.parametrize("act", OL.ACTS)
@pytest.mark.parametrize("form", FORMS)
def test_every_activation_in_every_form(hm, dev, form, act):
    for out in ("bf16", "f32"):
        p = _Product(hm, dev, form, act, 70, 96, 64, out, pad=2)
        p.call()
        p.check()


@pytest.mark.parametrize("form", FORMS)
def test_no_k(hm, dev, form):
    p = _Product(hm, dev, form, "gelu", 9, 37, 0, "bf16", pad=1)
    p.call()
    p.check()


@pytest.mark.parametrize("shape", [(3, 200, 512), (150, 384, 64), (700, 600, 256)])
@pytest.mark.parametrize("form", FORMS)
def test_outputs_over_inputs(hm, dev, shape, form):
    """D in its residual's, gate's or sum's place, out2 over the up product: the bits of separate outputs."""
    p = _Product(hm, dev, form, "gelu_tanh", *shape, "bf16")
    p.call()
    want, want2 = p.d.clone(), None if p.out2 is None else p.out2.clone()
    p.first[shape[0]] = 7.0
    p.d = p.first
    if form == "gated_gradient":
        p.second[shape[0]] = 7.0
        p.out2 = p.second
    p.call()
    m = shape[0]
    assert torch.equal(p.d[:m], want[:m]) and (want2 is None or torch.equal(p.out2[:m], want2[:m]))


def test_far_values(hm, dev):
    """Where an activation has flattened out its value and slope are the limits; NaN stays."""
    x = torch.tensor([-1e30, -300.0, -80.0, -20.0, 20.0, 300.0, 1e30, float("nan")], device=dev)
    one = torch.full((1, 32), 0x38, dtype=torch.uint8, device=dev)      # 1.0 in each of the 32 codes
    sa = torch.full((512,), 127 - 5, dtype=torch.uint8, device=dev)     # times 2^-5: the product is 1
    qb, sb = one.expand(8, 32).contiguous(), torch.full((512,), 127, dtype=torch.uint8, device=dev)
    d = torch.zeros(1, 8, device=dev)
    for act in range(1, 5):
        e = hm.hm_epilogue(hm.HM_EPI_GATED, act, 0, x.data_ptr(), 8, 0, 0, 0, 0)
        hm.mxfp8_gemm_epilogue(one.data_ptr(), 32, sa.data_ptr(), qb.data_ptr(), 32, sb.data_ptr(), 1, 8, 32, d.data_ptr(), 8, hm.HM_F32, e)
        v = d[0].tolist()
        assert max(abs(t) for t in v[:4]) < 5e-8 and np.allclose(v[4:7], [20.0, 300.0, 1e30], rtol=1e-6) and v[7] != v[7]
        e = hm.hm_epilogue(hm.HM_EPI_GRADIENT, act, 0, x.data_ptr(), 8, 0, 0, 0, 0)
        hm.mxfp8_gemm_epilogue(one.data_ptr(), 32, sa.data_ptr(), qb.data_ptr(), 32, sb.data_ptr(), 1, 8, 32, d.data_ptr(), 8, hm.HM_F32, e)
        v = d[0].tolist()
        assert max(abs(t) for t in v[:4]) < 5e-8 and np.allclose(v[4:7], 1.0, rtol=1e-6) and (act == 1 or v[7] != v[7])


# ---- quantization with the bias's gradient ------------------------------------
@pytest.mark.parametrize("rows,cols,block,pad", [(1, 33, 32, 0), (31, 128, 32, 0), (128, 1409, 128, 0), (129, 64, 32, 3),
                                                 (300, 257, 128, 5), (1025, 96, 32, 32), (5000, 130, 32, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("way", [(True, True), (False, True), (True, False)])
def test_quantize_bias(hm, dev, rows, cols, block, pad, dtype, way):
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols + pad)).astype(np.float32)).to(dev).to(_type(dtype))
    c32, r32 = -(-cols // 32) * 32, -(-rows // 32) * 32
    new = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device=dev)  # noqa: E731
    bufs = {}
    for name in ("plain", "bias"):
        bufs[name] = [new(rows, c32), new(hm.mxfp8_tiled_scale_bytes(rows, c32)), new(cols, r32), new(hm.mxfp8_tiled_scale_bytes(cols, r32))]
    ptrs = {k: ([v[0].data_ptr(), c32, v[1].data_ptr()] if way[0] else [0, 0, 0]) + ([v[2].data_ptr(), r32, v[3].data_ptr()] if way[1] else [0, 0, 0])
            for k, v in bufs.items()}
    ws = torch.full((max(16, hm.mxfp8_quantize_bias_workspace(rows, cols)),), 0xFF, dtype=torch.uint8, device=dev)
    db = torch.full((cols + 1,), 7.0, device=dev)
    hm.mxfp8_quantize(x.data_ptr(), _code(hm, x), rows, cols, cols + pad, 0, 0, block, *ptrs["plain"])
    hm.mxfp8_quantize_bias(x.data_ptr(), _code(hm, x), rows, cols, cols + pad, block, *ptrs["bias"], db.data_ptr(), False, ws.data_ptr(), ws.numel())
    assert all(torch.equal(a, b) for a, b in zip(bufs["plain"], bufs["bias"]))
    want = _np64(x)[:, :cols].sum(axis=0)
    tol = (70 + rows / 4096) * U * np.abs(_np64(x)[:, :cols]).sum(axis=0)
    once = _np64(db)
    assert (np.abs(once[:cols] - want) <= tol).all() and once[cols] == 7
    prior = torch.from_numpy(rng.standard_normal(cols).astype(np.float32)).to(dev)
    db[:cols] = prior
    hm.mxfp8_quantize_bias(x.data_ptr(), _code(hm, x), rows, cols, cols + pad, block, *ptrs["bias"], db.data_ptr(), True, ws.data_ptr(), ws.numel())
    assert np.array_equal(_np64(db)[:cols].astype(np.float32), (_np64(prior).astype(np.float32) + once[:cols].astype(np.float32)))


def test_quantize_bias_without_rows(hm, dev):
    db = torch.full((40,), 7.0, device=dev)
    q = torch.zeros(64, dtype=torch.uint8, device=dev)
    args = (0, hm.HM_F32, 0, 40, 40, 32, q.data_ptr(), 64, q.data_ptr(), 0, 0, 0, db.data_ptr())
    hm.mxfp8_quantize_bias(*args, True, 0, 0)
    assert (db == 7).all()
    hm.mxfp8_quantize_bias(*args, False, 0, 0)
    assert (db == 0).all()


# ---- heads -------------------------------------------------------------------
def _turns(dev, rot, theta=1e4):
    f, _ = OL.frequencies(rot, theta)
    t = [int(round(v / (2 * np.pi) * 2.0 ** 64)) for v in f]
    return f, torch.tensor(t, dtype=torch.int64, device=dev)


def _angles(positions, f):
    """Angles in 64 bits, whole turns dropped first in extended precision: positions to 2^40."""
    return np.asarray(np.mod(positions[:, None].astype(np.longdouble) * f[None].astype(np.longdouble), 2 * np.longdouble(np.pi)), dtype=np.float64)


class _Heads:
    """A packed projection's output [rows][pitch], its query and key heads and the outputs."""

    def __init__(self, hm, dev, rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew=0, far=5000, scale=1.0, seed=0):
        rng = np.random.default_rng(seed + rows + dim * 3 + rot)
        self.hm, self.rows, self.dim, self.rot, self.pairs, self.scale = hm, rows, dim, rot, pairs, scale
        self.eps, self.n = 1e-5, (hq, hk)
        dt = _type(dtype)
        put = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(dt)  # noqa: E731
        pitch = (hq + 2 * hk) * dim + skew
        self.packed = put(rows * pitch + skew)[skew:]
        self.pitch = pitch
        self.pos = rng.integers(-far, far + 1, rows)
        self.pos[-1] = far
        self.tpos = torch.from_numpy(self.pos).to(dev)
        self.f, self.turns = _turns(dev, rot) if rot else (np.zeros(0), torch.zeros(1, dtype=torch.int64, device=dev))
        self.gamma = [torch.from_numpy(rng.uniform(0.5, 1.5, dim).astype(np.float32)).to(dev) if norm else None for _ in range(2)]
        self.out = [self._matrix(torch.full((h * rows * dim + skew + 1,), 7.0, dtype=dt, device=dev), h, place, skew) for h in self.n]
        self.dy = [self._matrix(put(h * rows * dim + skew + 1), h, place, skew) for h in self.n]
        self.dx = torch.full((rows * pitch + 1,), 7.0, dtype=dt, device=dev)
        self.dgamma = [torch.full((dim,), 3.0, device=dev) for _ in range(2)]

    def _matrix(self, flat, heads, place, skew):
        """(tensor, offset, row stride, head stride)"""
        return (flat, skew, self.dim if place == "heads" else heads * self.dim, self.rows * self.dim if place == "heads" else self.dim)

    def view(self, m, heads):
        return torch.as_strided(m[0], (self.rows, heads, self.dim), (m[2], m[3], 1), m[1] + m[0].storage_offset())

    def x(self, g):
        first = 0 if g == 0 else self.n[0]
        return (self.packed, first * self.dim, self.pitch, self.dim)

    def grad(self, g):
        first = 0 if g == 0 else self.n[0]
        return (self.dx, first * self.dim, self.pitch, self.dim)

    @staticmethod
    def _at(m):
        return (m[0].data_ptr() + m[1] * m[0].element_size(), m[2], m[3])

    def rotation(self):
        hm = self.hm
        return hm.hm_rotation(self.turns.data_ptr(), self.tpos.data_ptr(), self.scale, self.rot, hm.HM_ROPE_PAIRS if self.pairs else hm.HM_ROPE_HALF)

    def forward(self, outs=None, stream=0):
        outs = outs or self.out
        groups = self.hm.head_list([(*self._at(self.x(g)), *self._at(outs[g]), self.gamma[g].data_ptr() if self.gamma[g] is not None else 0,
                                     self.n[g]) for g in range(2)])
        self.hm.head_norm_rope(groups, _code(self.hm, self.packed), self.rows, self.dim, self.eps, self.rotation(), stream)

    def backward(self, dys=None, dxs=None, accumulate=False, stream=0):
        hm = self.hm
        dys, dxs = dys or self.dy, dxs or [self.grad(0), self.grad(1)]
        groups = hm.head_grad_list([(*self._at(dys[g]), *self._at(self.x(g)), *self._at(dxs[g]),
                                     self.gamma[g].data_ptr() if self.gamma[g] is not None else 0,
                                     self.dgamma[g].data_ptr() if self.gamma[g] is not None else 0, self.n[g], accumulate) for g in range(2)])
        need = hm.head_norm_rope_backward_workspace(groups, self.rows, self.dim)
        self.ws = torch.full((max(16, need),), 0xFF, dtype=torch.uint8, device=self.packed.device)
        hm.head_norm_rope_backward(groups, _code(hm, self.packed), self.rows, self.dim, self.eps, self.rotation(), self.ws.data_ptr(),
                                   self.ws.numel(), stream)

    def pair_sum(self, v):
        """|a| + |b| of each element's pair, times the scale; |v| past the rotated part."""
        v = np.abs(v)
        out = v.copy()
        if self.rot:
            i = np.arange(self.rot // 2)
            a, b = (2 * i, 2 * i + 1) if self.pairs else (i, i + self.rot // 2)
            out[..., a] = out[..., b] = self.scale * (v[..., a] + v[..., b])
        return out

    def near(self, got, want, tol):
        tol = tol + 2 * U * np.abs(want)
        if self.packed.dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        err = np.abs(got - want)
        assert np.isfinite(err).all() and (err <= tol + 1e-37).all(), f"worst excess {np.max(err / (tol + 1e-37))}"

    def check_forward(self, outs=None, x=None):
        for g in range(2):
            x_g = _np64(self.view(self.x(g), self.n[g])) if x is None else x[g]
            gamma = None if self.gamma[g] is None else _np64(self.gamma[g])
            a = _angles(self.pos, self.f)
            v = OL.heads(x_g, gamma, self.eps, a[:, :0], 1.0, False)
            got = _np64(self.view((outs or self.out)[g], self.n[g]))
            self.near(got, OL.turn(v, a, self.scale, self.pairs), 24 * U * self.pair_sum(v))

    def check_backward(self, dys=None, dxs=None, times=1):
        a = _angles(self.pos, self.f)
        for g in range(2):
            x, dy = _np64(self.view(self.x(g), self.n[g])), _np64(self.view((dys or self.dy)[g], self.n[g]))
            gamma = None if self.gamma[g] is None else _np64(self.gamma[g])
            dx, dgamma = OL.heads_grad(dy, x, gamma, self.eps, a, self.scale, self.pairs)
            t = self.pair_sum(dy)
            got = _np64(self.view((dxs or [self.grad(0), self.grad(1)])[g], self.n[g]))
            if gamma is None:
                self.near(got, dx, 24 * U * t)
                continue
            r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + self.eps)
            xhat, u = np.abs(x * r), t * np.abs(gamma)
            self.near(got, dx, 96 * U * r * (u + xhat * np.mean(u * xhat, axis=-1, keepdims=True)))
            tol = (self.rows * self.n[g] + 88) * U * (t * xhat).sum(axis=(0, 1))
            assert (np.abs(_np64(self.dgamma[g]) - times * dgamma) <= times * tol + 1e-37).all()


HEADS = [
    # rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew
    (1, 32, 8, 128, 128, False, True, "bf16", "rows", 0),
    (1, 1, 1, 32, 32, True, True, "f32", "heads", 0),
    (3, 4, 4, 64, 64, False, True, "bf16", "heads", 0),
    (70, 40, 40, 128, 128, False, True, "bf16", "heads", 0),
    (33, 32, 8, 128, 64, True, True, "f32", "rows", 0),
    (515, 12, 3, 80, 24, True, False, "f32", "rows", 0),
    (129, 5, 1, 96, 96, False, True, "bf16", "rows", 0),
    (40, 3, 2, 72, 72, False, True, "bf16", "heads", 0),
    (40, 3, 2, 72, 18, True, True, "f32", "rows", 0),
    (21, 2, 2, 80, 40, True, True, "bf16", "rows", 0),
    (21, 2, 2, 80, 20, False, True, "bf16", "heads", 0),
    (17, 2, 1, 192, 96, False, True, "bf16", "rows", 0),
    (17, 2, 1, 256, 256, True, True, "f32", "heads", 0),
    (9, 2, 1, 512, 512, False, True, "bf16", "rows", 0),
    (9, 2, 1, 512, 500, True, True, "f32", "rows", 0),
    (9, 2, 1, 510, 510, False, True, "bf16", "rows", 0),
    (50, 3, 1, 128, 128, False, True, "bf16", "rows", 1),     # addresses and pitches of no vector
    (50, 3, 1, 128, 128, True, True, "f32", "heads", 1),
    (50, 3, 1, 128, 64, True, False, "bf16", "rows", 2),
    (50, 3, 1, 64, 64, False, True, "f32", "rows", 4),
    (11, 2, 1, 2, 2, False, True, "bf16", "rows", 0),
    (11, 2, 1, 6, 2, True, True, "f32", "rows", 0),
    (200, 7, 5, 128, 0, False, True, "bf16", "rows", 0),      # the norm alone
    (2000, 4, 1, 64, 32, False, True, "bf16", "rows", 0),
    (4, 1, 1, 32, 32, False, False, "bf16", "rows", 0),
]


@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
def test_heads(hm, dev, case):
    rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew = case
    h = _Heads(hm, dev, rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew, scale=1.25 if rows % 2 else 1.0)
    before = h.packed.clone()
    h.forward()
    h.check_forward()
    for flat, at, *_ in h.out:
        assert (flat[:at] == 7).all() and flat[-1] == 7
    assert torch.equal(before, h.packed)


@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
def test_heads_gradient(hm, dev, case):
    rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew = case
    h = _Heads(hm, dev, rows, hq, hk, dim, rot, pairs, norm, dtype, place, skew, scale=1.25 if rows % 2 else 1.0)
    h.backward()
    h.check_backward()
    # the values' columns, the pitch's rest and the guard stay as they were
    rest = h.dx[:rows * h.pitch].view(rows, h.pitch)[:, (hq + hk) * dim:]
    assert (rest == 7).all() and h.dx[-1] == 7
    if norm:
        first = [t.clone() for t in h.dgamma]
        h.backward(accumulate=True)
        assert all(torch.equal(t, f + f) for t, f in zip(h.dgamma, first))
        h.check_backward(times=2)


@pytest.mark.parametrize("far", [1000000, 2 ** 31 + 12345, 2 ** 40])
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(hm, dev, far, pairs):
    """The angle's fraction of a turn is exact to pos 2^-65 turns, whatever the position; the
    frequency's own rounding to 2^-64 turns is the table's, so the oracle takes the table's value."""
    h = _Heads(hm, dev, 64, 4, 2, 64, 64, pairs, True, "f32", "rows", far=far)
    h.f = np.array([int(t) for t in h.turns.tolist()], dtype=np.longdouble) / np.longdouble(2.0 ** 64)
    turn = lambda p: np.array([[(int(q) * int(t)) % 2 ** 64 / 2.0 ** 64 for t in h.turns.tolist()] for q in p])  # noqa: E731
    a = 2 * np.pi * turn(h.pos)
    h.forward()
    for g in range(2):
        v = OL.heads(_np64(h.view(h.x(g), h.n[g])), _np64(h.gamma[g]), h.eps, a[:, :0], 1.0, False)
        h.near(_np64(h.view(h.out[g], h.n[g])), OL.turn(v, a, 1.0, pairs), 24 * U * h.pair_sum(v))


@pytest.mark.parametrize("dtype,dim,rot,pairs,skew", [("bf16", 128, 128, False, 0), ("f32", 80, 20, True, 0), ("bf16", 64, 64, True, 1)])
def test_in_place(hm, dev, dtype, dim, rot, pairs, skew):
    """Queries and keys turned where they stand in the packed rows; values and gaps stay."""
    h = _Heads(hm, dev, 37, 6, 2, dim, rot, pairs, True, dtype, "rows", skew)
    x = [_np64(h.view(h.x(g), h.n[g])) for g in range(2)]
    rows = h.packed[:37 * h.pitch].view(37, h.pitch)
    rest = rows[:, 8 * dim:].clone()
    places = [h.x(0), h.x(1)]
    h.forward(places)
    h.check_forward(places, x)
    assert torch.equal(rows[:, 8 * dim:], rest)
    # the gradient over dy
    h2 = _Heads(hm, dev, 37, 6, 2, dim, rot, pairs, True, dtype, "rows", skew)
    kept = [(m[0].clone(), *m[1:]) for m in h2.dy]
    h2.backward(dxs=h2.dy)
    h2.check_backward(dys=kept, dxs=h2.dy)


def test_broadcast_gradient(hm, dev):
    """dy with strides of zero: one row for all rows and heads, as a sum's gradient arrives."""
    h = _Heads(hm, dev, 45, 4, 2, 64, 64, False, True, "f32", "rows")
    one = torch.randn(64, device=dev)
    dys = [(one, 0, 0, 0), (one, 0, 0, 0)]
    h.backward(dys=dys)
    h.check_backward(dys=dys)


def test_heads_without_gamma_gradient_and_without_rows(hm, dev):
    h = _Heads(hm, dev, 20, 2, 2, 64, 64, False, True, "f32", "rows")
    x, dy, dx = (h._at(m) for m in (h.x(0), h.dy[0], h.grad(0)))
    frozen = hm.head_grad_list([(*dy, *x, *dx, h.gamma[0].data_ptr(), 0, 2, False)])
    assert hm.head_norm_rope_backward_workspace(frozen, 20, 64) == 0
    hm.head_norm_rope_backward(frozen, hm.HM_F32, 20, 64, h.eps, h.rotation(), 0, 0)
    alone = h.dx.clone()
    h.backward()
    cols = slice(0, 128)
    assert torch.equal(alone[:20 * h.pitch].view(20, -1)[:, cols], h.dx[:20 * h.pitch].view(20, -1)[:, cols])
    for acc, want in ((True, 3.0), (False, 0.0)):
        dg = torch.full((64,), 3.0, device=dev)
        none = hm.head_grad_list([(0, 0, 0, 0, 0, 0, 0, 0, 0, h.gamma[0].data_ptr(), dg.data_ptr(), 2, acc)])
        hm.head_norm_rope_backward(none, hm.HM_F32, 0, 64, h.eps, h.rotation(), 0, 0)
        assert (dg == want).all()
    # a group without heads beside one with: its sum is empty
    dg = torch.full((64,), 3.0, device=dev)
    two = hm.head_grad_list([(0, 0, 0, 0, 0, 0, 0, 0, 0, h.gamma[0].data_ptr(), dg.data_ptr(), 0, False),
                             (*dy, *x, *dx, h.gamma[0].data_ptr(), h.dgamma[0].data_ptr(), 2, False)])
    want = h.dgamma[0].clone()
    ws = torch.zeros(max(16, hm.head_norm_rope_backward_workspace(two, 20, 64)), dtype=torch.uint8, device=dev)
    hm.head_norm_rope_backward(two, hm.HM_F32, 20, 64, h.eps, h.rotation(), ws.data_ptr(), ws.numel())
    assert (dg == 0).all() and torch.allclose(h.dgamma[0], want, rtol=1e-5)


def test_special_values_stay_in_their_head(hm, dev):
    h = _Heads(hm, dev, 6, 4, 2, 64, 64, False, True, "f32", "rows")
    clean = h.packed.clone()
    h.forward()
    want = [m[0].clone() for m in h.out]
    v = h.view(h.x(0), 4)
    v[2, 1, 5] = float("nan")
    v[3, 0, 7] = float("inf")
    v[4, 2] = 0.0
    h.forward()
    got, ref = h.view(h.out[0], 4), torch.as_strided(want[0], (6, 4, 64), (h.out[0][2], h.out[0][3], 1), h.out[0][1])
    assert torch.isnan(got[2, 1]).all() and torch.isnan(got[3, 0]).any() and (got[4, 2] == 0).all()
    same = torch.ones(6, 4, dtype=torch.bool)
    same[2, 1] = same[3, 0] = same[4, 2] = False
    assert torch.equal(got[same.to(dev)], ref[same.to(dev)]) and torch.equal(h.out[1][0], want[1])
    h.packed.copy_(clean)


def test_replay_and_two_streams(hm, dev):
    """All of them captured, replayed on other inputs, and run on two streams at once: the bits of
    calls made one by one."""
    def work(seed):
        p = _Product(hm, dev, "forward", "gelu", 150, 256, 128, "bf16", seed=seed)
        g = _Product(hm, dev, "gated_gradient", "silu", 40, 320, 512, "f32", seed=seed)
        h = _Heads(hm, dev, 90, 8, 2, 64, 64, False, True, "bf16", "heads", seed=seed)
        q = [torch.zeros(n, dtype=torch.uint8, device=dev) for n in (150 * 256, hm.mxfp8_tiled_scale_bytes(150, 256), 256 * 160,
                                                                      hm.mxfp8_tiled_scale_bytes(256, 160), hm.mxfp8_quantize_bias_workspace(150, 256))]
        db = torch.zeros(256, device=dev)

        def step():
            st = torch.cuda.current_stream().cuda_stream
            p.call(st)
            hm.mxfp8_quantize_bias(p.d.data_ptr(), hm.HM_BF16, 150, 256, 256, 32, q[0].data_ptr(), 256, q[1].data_ptr(), q[2].data_ptr(), 160,
                                   q[3].data_ptr(), db.data_ptr(), False, q[4].data_ptr(), q[4].numel(), st)
            g.call(st)
            h.forward(stream=st)
            h.backward(stream=st)
        outs = [p.d, p.out2, *q[:4], db, g.d, g.out2, h.out[0][0], h.out[1][0], h.dx, *h.dgamma]
        ins = [p.qa, p.first, g.qb, g.second, h.packed, h.tpos]
        return step, outs, ins

    step, outs, ins = work(0)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other, outs2, ins2 = work(50)
    for a, b in zip(ins, ins2):
        a.copy_(b)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.fill_(7)  # the guards' own value
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    other()
    torch.cuda.synchronize()
    want2 = [t.clone() for t in outs2]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for t in outs + outs2:
            t.fill_(7)  # the guards' own value
        torch.cuda.synchronize()
        for s, f in ((s1, step), (s2, other)):
            with torch.cuda.stream(s):
                f()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + outs2, want + want2))
    assert hm.hm_device_error() == 0


@pytest.mark.parametrize("extra,dim", [(0, 32), (1, 32), (0, 16), (0, 512)])
def test_many_rows_per_cta(hm, dev, extra, dim):
    """Rows that leave some CTAs 1024 each, which fit beside the angles, and others one more, which
    do not: forward and gradient, one head of each kind, every row compared.  Angles of one head's
    rows, 1024 positions and the rings together are the most that a CTA asks for."""
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    g = torch.Generator(device=dev)
    g.manual_seed(extra)
    for ctas, back in ((4 * sms // 2, False), (2 * sms // 2, True)):
        rows = 1024 * ctas + extra
        x = torch.randn(rows, 2, dim, generator=g, device=dev).bfloat16()
        dy = torch.randn(rows, 2, dim, generator=g, device=dev).bfloat16()
        pos = torch.randint(0, 100000, (rows,), generator=g, device=dev)
        f, turns = _turns(dev, dim)
        gamma = torch.rand(dim, generator=g, device=dev) + 0.5
        out = torch.full((rows + 1, 2, dim), 7.0, device=dev, dtype=torch.bfloat16)
        dg = torch.zeros(2, dim, device=dev)
        rot = hm.hm_rotation(turns.data_ptr(), pos.data_ptr(), 1.0, dim, hm.HM_ROPE_HALF)
        at = lambda t, h: (t.data_ptr() + 2 * h * dim, 2 * dim, dim)  # noqa: E731
        a = pos.double()[:, None, None] * torch.from_numpy(f).to(dev)
        x64 = x.double().requires_grad_()
        v = x64 * torch.rsqrt(x64.square().mean(-1, keepdim=True) + 1e-5) * gamma.double()
        u, w = v[..., :dim // 2], v[..., dim // 2:]
        y = torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], -1)
        if back:
            lst = hm.head_grad_list([(*at(dy, h), *at(x, h), *at(out, h), gamma.data_ptr(), dg[h].data_ptr(), 1, False) for h in range(2)])
            ws = torch.empty(hm.head_norm_rope_backward_workspace(lst, rows, dim), dtype=torch.uint8, device=dev)
            hm.head_norm_rope_backward(lst, hm.HM_BF16, rows, dim, 1e-5, rot, ws.data_ptr(), ws.numel())
            want, = torch.autograd.grad((y * dy.double()).sum(), x64)
        else:
            hm.head_norm_rope(hm.head_list([(*at(x, h), *at(out, h), gamma.data_ptr(), 1) for h in range(2)]), hm.HM_BF16, rows, dim, 1e-5, rot)
            want = y.detach()
        assert (out[rows] == 7).all()
        # half a bf16 step and the bounds of heads and gradient with each term at its head's largest
        r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-5)
        most = (96 * r * 3 * (1 + dim ** 0.5) * dy.double().abs().amax(-1, keepdim=True) if back
                else 48 * v.detach().abs().amax(-1, keepdim=True))
        err = (out[:rows].double() - want).abs()
        assert bool((err <= (1 + 2.0 ** -8) * U * most + 2.0 ** -8 * want.abs()).all())


def test_more_than_two_groups(hm, dev):
    """Four groups of one call: the bits of four calls; their gammas' gradients to their sums' order."""
    rows, dim = 150, 64
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    heads = (5, 2, 1, 3)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, dy = [rand(rows, h, dim) for h in heads], [rand(rows, h, dim) for h in heads]
    gamma = [rand(dim), None, rand(dim), rand(dim)]
    pos = torch.randint(0, 9000, (rows,), generator=g, device=dev)
    _, turns = _turns(dev, dim)
    rot = hm.hm_rotation(turns.data_ptr(), pos.data_ptr(), 1.0, dim, hm.HM_ROPE_PAIRS)
    p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    at = lambda t: (t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731

    def run(parts):
        y, dx = [torch.zeros_like(t) for t in x], [torch.zeros_like(t) for t in x]
        dg = [torch.zeros(dim, device=dev) for _ in x]
        for part in parts:
            hm.head_norm_rope(hm.head_list([(*at(x[i]), *at(y[i]), p(gamma[i]), heads[i]) for i in part]), hm.HM_F32, rows, dim, 1e-6, rot)
            lst = hm.head_grad_list([(*at(dy[i]), *at(x[i]), *at(dx[i]), p(gamma[i]), p(dg[i]) if gamma[i] is not None else 0, heads[i], False)
                                     for i in part])
            ws = torch.empty(max(16, hm.head_norm_rope_backward_workspace(lst, rows, dim)), dtype=torch.uint8, device=dev)
            hm.head_norm_rope_backward(lst, hm.HM_F32, rows, dim, 1e-6, rot, ws.data_ptr(), ws.numel())
        return y, dx, dg

    y, dx, dg = run([range(4)])
    y1, dx1, dg1 = run([[0], [1], [2], [3]])
    assert all(torch.equal(a, b) for a, b in zip(y + dx, y1 + dx1))
    assert all(float((a - b).abs().max()) <= 2 * (rows * 5 + 88) * U * float(t.abs().sum()) for a, b, t in zip(dg, dg1, dy))


def test_a_wait_that_gives_up_in_an_epilogue_kernel(hm, dev, monkeypatch):
    """The accumulator is never signalled (a switch of the launch): the bounded waits run out, the error is
    reported once, and the next product is right."""
    monkeypatch.setenv("HM_INJECT_MX_WAIT_TIMEOUT", "1")
    for shape in ((9, 130, 96), (700, 3000, 256)):
        p = _Product(hm, dev, "gated_gradient", "silu", *shape, "bf16")
        monkeypatch.setenv("HM_INJECT_MX_WAIT_TIMEOUT", "1")
        p.call()
        torch.cuda.synchronize()
        assert hm.hm_device_error() == hm.HM_ERR_TIMEOUT
        monkeypatch.setenv("HM_INJECT_MX_WAIT_TIMEOUT", "0")
        p.call()
        p.check()
        assert hm.hm_device_error() == 0
