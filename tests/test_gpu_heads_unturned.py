"""Elements past the rotated part of a head stay out of the rotation, whatever they hold:
an infinity or NaN among them reaches neither its neighbours nor the turned pairs except
through the norm, forward and backward, at every vector width of the kernels.

Without gamma they are copied, bit for bit.  With gamma the norm's root of an infinite mean is
infinite: 0 for every finite element, NaN for the infinite one, as in 64 bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layers as OL  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROWS, HEADS = 13, 3
# dtype, dim, rot, pairs, elements off alignment: vectors of 8, 4, 2 and 1 elements
KINDS = [("bf16", 128, 64, False, 0), ("bf16", 128, 32, True, 0), ("bf16", 80, 40, True, 0), ("bf16", 72, 36, False, 0), ("bf16", 72, 18, True, 0),
         ("bf16", 72, 18, False, 1), ("f32", 96, 32, False, 0), ("f32", 80, 24, True, 0), ("f32", 12, 4, False, 0), ("f32", 10, 2, True, 0),
         ("f32", 34, 18, False, 1), ("f32", 512, 2, False, 0)]


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


class _Case:
    def __init__(self, hm, dev, dtype, dim, rot, pairs, skew):
        self.hm, self.dim, self.rot, self.pairs = hm, dim, rot, pairs
        self.dt, self.code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
        g = torch.Generator(device=dev)
        g.manual_seed(dim + rot)
        self.new = lambda: torch.randn(ROWS * HEADS * dim + skew, generator=g, device=dev).to(self.dt)[skew:].view(ROWS, HEADS, dim)  # noqa: E731
        self.x, self.dy, self.out = self.new(), self.new(), self.new()
        self.gamma = torch.rand(dim, generator=g, device=dev) + 0.5
        self.dgamma = torch.zeros(dim, device=dev)
        self.pos = torch.randint(1, 5000, (ROWS,), generator=g, device=dev)
        turns, _ = hm.rope_turns(rot)
        self.turns = torch.tensor(turns, dtype=torch.int64, device=dev)
        # the table's own frequencies, whole turns dropped in integers
        self.angles = 2 * np.pi * np.array([[(p * t) % 2 ** 64 / 2.0 ** 64 for t in turns] for p in self.pos.tolist()])
        self.rotation = hm.hm_rotation(self.turns.data_ptr(), self.pos.data_ptr(), 1.0, rot, hm.HM_ROPE_PAIRS if pairs else hm.HM_ROPE_HALF)

    def at(self, t):
        return t.data_ptr(), t.stride(0), t.stride(1)

    def forward(self, norm):
        g = self.gamma.data_ptr() if norm else 0
        self.hm.head_norm_rope(self.hm.head_list([(*self.at(self.x), *self.at(self.out), g, HEADS)]), self.code, ROWS, self.dim, 1e-5, self.rotation)

    def backward(self, norm):
        g, dg = (self.gamma.data_ptr(), self.dgamma.data_ptr()) if norm else (0, 0)
        lst = self.hm.head_grad_list([(*self.at(self.dy), *self.at(self.x), *self.at(self.out), g, dg, HEADS, False)])
        ws = torch.empty(max(16, self.hm.head_norm_rope_backward_workspace(lst, ROWS, self.dim)), dtype=torch.uint8, device=self.x.device)
        self.hm.head_norm_rope_backward(lst, self.code, ROWS, self.dim, 1e-5, self.rotation, ws.data_ptr(), ws.numel())


def _np(t):
    return t.detach().cpu().double().numpy()


def _spoil(c, t):
    """An infinity or NaN at each place past the rotated part in turn, its neighbours finite."""
    past = range(c.rot, c.dim)
    values = (float("inf"), float("-inf"), float("nan"))
    for i in range(ROWS * HEADS - 4):  # the last heads stay clean
        t[i // HEADS, i % HEADS, past[i * 5 % len(past)]] = values[i % 3]


def _same(got, want, tol):
    """NaN where `want` is, the same infinities, the finite values to `tol`."""
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert (np.abs(got - want)[finite] <= tol[finite] + 1e-37).all()


def _pair_sum(c, v):
    """|a| + |b| of each element's pair; |v| past the rotated part."""
    i = np.arange(c.rot // 2)
    a, b = (2 * i, 2 * i + 1) if c.pairs else (i, i + c.rot // 2)
    out = np.abs(v)
    out[..., a] = out[..., b] = out[..., a] + out[..., b]
    return out


def _rounded(c, tol, want):
    """With the output's rounding: half a step, 2^-8 or 2^-24 of it."""
    return tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) if c.dt == torch.bfloat16 else tol + U * np.abs(want)


@pytest.mark.parametrize("kind", KINDS, ids=lambda c: "-".join(map(str, c)))
def test_copied_without_gamma(hm, dev, kind):
    c = _Case(hm, dev, *kind)
    bits = torch.int16 if c.dt == torch.bfloat16 else torch.int32
    for call, source in ((c.forward, c.x), (c.backward, c.dy)):
        c.out.copy_(source)
        call(False)
        clean = c.out.clone()
        source[0, 0, c.rot:] = -0.0
        _spoil(c, source)
        call(False)
        past, want = c.out[..., c.rot:], source[..., c.rot:]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(past), nan)
        assert torch.equal(past[~nan].view(bits), want[~nan].view(bits))
        assert torch.equal(c.out[..., :c.rot], clean[..., :c.rot])


@pytest.mark.parametrize("kind", KINDS, ids=lambda c: "-".join(map(str, c)))
def test_forward_with_gamma(hm, dev, kind):
    c = _Case(hm, dev, *kind)
    _spoil(c, c.x)
    c.forward(True)
    with np.errstate(invalid="ignore"):
        v = OL.heads(_np(c.x), _np(c.gamma), 1e-5, c.angles[:, :0], 1.0, False)
        want = v.copy()
        # the rotated pairs alone: in a complex product NaN would spread by itself
        want[..., :c.rot] = OL.turn(v[..., :c.rot], c.angles, 1.0, c.pairs)
        _same(_np(c.out), want, _rounded(c, 24 * U * _pair_sum(c, v), want))


@pytest.mark.parametrize("kind", KINDS, ids=lambda c: "-".join(map(str, c)))
def test_gradient_with_gamma(hm, dev, kind):
    """dy spoiled past the rotated part: the head's dx through its mean, dgamma at those columns alone."""
    c = _Case(hm, dev, *kind)
    past = c.rot + (c.dim - c.rot) // 3
    c.dy[4, 1, past] = float("inf")
    c.backward(True)
    x, dy, gamma = _np(c.x), _np(c.dy), _np(c.gamma)
    with np.errstate(invalid="ignore"):
        t = dy.copy()
        t[..., :c.rot] = OL.turn(dy[..., :c.rot], c.angles, 1.0, c.pairs, back=True)
        r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + 1e-5)
        xhat, u = x * r, t * gamma
        dx = r * (u - xhat * np.mean(u * xhat, axis=-1, keepdims=True))
        dgamma = (t * xhat).sum(axis=(0, 1))
        T = _pair_sum(c, dy)
        ua = T * gamma
        tol = 96 * U * r * (ua + np.abs(xhat) * np.mean(ua * np.abs(xhat), axis=-1, keepdims=True))
        _same(_np(c.out), dx, _rounded(c, tol, dx))
        _same(_np(c.dgamma), dgamma, (ROWS * HEADS + 88) * U * (T * np.abs(xhat)).sum(axis=(0, 1)))
    assert np.isfinite(_np(c.dgamma)).sum() == c.dim - 1
