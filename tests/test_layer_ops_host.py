"""Refusals of the operators of a layer's projections, and the rotation's
frequencies: all on the host before anything is launched.  Addresses are never
dereferenced."""
import numpy as np
import pytest

from oracle import layers as OL

A, B, S1, S2, D, W, X, Y = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(8))
GRAD = dict(form=2, bias=0, in_=X)
GATED_GRAD = dict(form=3, bias=0, in_=X, in2=Y, out2=W)


def _status(fn, *args):
    try:
        fn(*args)
    except Exception as e:
        return e.status
    return 0


def _is(hm, got, status):
    assert got == (0 if status == "OK" else getattr(hm, "HM_ERR_" + status))


def _gemm(hm, **kw):
    v = dict(a=A, lda=64, sa=S1, b=B, ldb=64, sb=S2, m=5, n=7, k=64, d=D, ldd=7, t=hm.HM_BF16)
    e = dict(form=0, act=1, bias=W + 4096, in_=0, ld_in=7, in2=0, ld_in2=7, out2=0, ld_out2=7)
    for k, x in kw.items():
        (v if k in v else e)[k] = x
    return _status(hm.mxfp8_gemm_epilogue, *v.values(), hm.hm_epilogue(*e.values()))


@pytest.mark.parametrize("kw,status", [
    (dict(form=-1), "ARG"), (dict(form=4), "ARG"), (dict(act=-1), "ARG"), (dict(act=5), "ARG"),
    (dict(m=-1), "ARG"), (dict(a=0), "ARG"), (dict(d=0), "ARG"), (dict(ldd=6), "ARG"), (dict(t=0), "DTYPE"),
    (dict(k=48), "ALIGN"), (dict(lda=72), "ALIGN"), (dict(d=D + 1), "ALIGN"), (dict(bias=W + 2), "ALIGN"),
    (dict(in_=X + 1), "ALIGN"), (dict(out2=X + 1), "ALIGN"), (dict(t=2, in_=X + 2), "ALIGN"),
    (dict(in_=X, ld_in=6), "ARG"), (dict(out2=X, ld_out2=6), "ARG"), (dict(in2=X), "ARG"),     # forward takes no in2
    (dict(form=1), "ARG"), (dict(form=1, in_=X, in2=Y), "ARG"),                                # the gate is needed
    (dict(form=2, in_=X), "ARG"), (dict(form=2, bias=0), "ARG"), (dict(GRAD, out2=Y), "ARG"),  # no bias, no out2
    (dict(GATED_GRAD, in2=0), "ARG"), (dict(GATED_GRAD, out2=0), "ARG"), (dict(GATED_GRAD, bias=W), "ARG"),
    (dict(GATED_GRAD, ld_in2=6), "ARG"), (dict(in_=X, ld_in=2 ** 41), "GEOMETRY"), (dict(m=2 ** 31), "GEOMETRY"),
    (dict(d=A), "OVERLAP"), (dict(out2=A), "OVERLAP"), (dict(out2=S2 + 16), "OVERLAP"), (dict(out2=D), "OVERLAP"),
    (dict(out2=D + 4), "OVERLAP"), (dict(d=W + 4096), "OVERLAP"), (dict(out2=W + 4100), "OVERLAP"),
    (dict(in_=D + 2), "OVERLAP"), (dict(in_=D, ld_in=8), "OVERLAP"), (dict(GATED_GRAD, in2=D + 14), "OVERLAP"),
    (dict(GATED_GRAD, out2=X + 14), "OVERLAP"), (dict(m=0), "OK"), (dict(n=0, bias=0), "OK"), (dict(m=0, d=0, a=0), "OK"),
])
def test_epilogue_refusals(hm, kw, status):
    _is(hm, _gemm(hm, **kw), status)


def test_epilogue_is_needed(hm):
    assert hm.lib().mxfp8_gemm_epilogue(A, 64, S1, B, 64, S2, 5, 7, 64, D, 7, hm.HM_BF16, None, None) == hm.HM_ERR_ARG


def _bias(hm, **kw):
    v = dict(x=A, t=hm.HM_BF16, rows=140, cols=70, ldx=70, block=32, q=B, ldq=96, s=S1, qt=D, ldqt=160, st=S2, db=W,
             acc=False, ws=X, ws_bytes=2 * 70 * 4)
    v.update(kw)
    return _status(hm.mxfp8_quantize_bias, *v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(cols=-1), "ARG"), (dict(block=64), "ARG"), (dict(x=0), "ARG"), (dict(db=0), "ARG"),
    (dict(q=0), "ARG"), (dict(qt=0), "ARG"), (dict(q=0, s=0, qt=0, st=0), "ARG"), (dict(ldqt=128), "ARG"),
    (dict(db=W + 2), "ALIGN"), (dict(ws=X + 8), "ALIGN"), (dict(x=A + 1), "ALIGN"), (dict(t=0), "DTYPE"),
    (dict(ws=0), "WORKSPACE"), (dict(ws_bytes=2 * 70 * 4 - 1), "WORKSPACE"), (dict(rows=2 ** 22 + 1), "GEOMETRY"),
    (dict(cols=2 ** 30 + 1), "GEOMETRY"), (dict(db=A), "OVERLAP"), (dict(db=S1), "OVERLAP"), (dict(ws=D), "OVERLAP"),
    (dict(ws=A + 16), "OVERLAP"), (dict(db=X + 4), "OVERLAP"), (dict(db=B + 4), "OVERLAP"), (dict(cols=0, db=0), "OK"),
    (dict(rows=0, acc=True), "OK"), (dict(cols=0), "OK"),
])
def test_quantize_bias_refusals(hm, kw, status):
    _is(hm, _bias(hm, **kw), status)


def test_quantize_bias_workspace(hm):
    assert hm.mxfp8_quantize_bias_workspace(128, 4096) == 0
    assert hm.mxfp8_quantize_bias_workspace(129, 33) == 2 * 33 * 4
    assert _status(hm.mxfp8_quantize_bias_workspace, -1, 3) == hm.HM_ERR_ARG
    assert _status(hm.mxfp8_quantize_bias_workspace, 2 ** 22 + 1, 3) == hm.HM_ERR_GEOMETRY


def _rotation(hm, kw):
    r = dict(turns=S1, positions=S2, scale=1.0, rot=16, layout=0)
    for k in list(r):
        if k in kw:
            r[k] = kw.pop(k)
    return hm.hm_rotation(*r.values())


def _heads(hm, **kw):
    rot = _rotation(hm, kw)
    g = dict(x=A, x_row=96, x_head=16, y=B, y_row=64, y_head=16, gamma=D, heads=4)
    v = dict(t=hm.HM_BF16, rows=3, dim=16, eps=1e-6)
    two = kw.pop("two", None)
    for k, x in kw.items():
        (g if k in g else v)[k] = x
    groups = [tuple(g.values())] + ([tuple({**g, **two}.values())] if two else [])
    return _status(hm.head_norm_rope, hm.head_list(groups), v["t"], v["rows"], v["dim"], v["eps"], rot, 0)


KEYS = dict(x=A + 4 * 32, y=B + 2 ** 20, heads=2)  # behind the queries of each row of the packed projection


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(dim=-2), "ARG"), (dict(eps=-1.0), "ARG"), (dict(eps=float("nan")), "ARG"),
    (dict(x=0), "ARG"), (dict(y=0), "ARG"), (dict(heads=-1), "ARG"), (dict(x_row=-1), "ARG"), (dict(x_head=-16), "ARG"),
    (dict(y_head=15), "ARG"), (dict(y_row=63), "ARG"), (dict(y_row=15, y_head=1000), "ARG"),
    (dict(y_row=16, y_head=47), "ARG"), (dict(layout=2), "ARG"), (dict(scale=float("inf")), "ARG"),
    (dict(scale=float("nan")), "ARG"), (dict(rot=-2), "ARG"), (dict(turns=0), "ARG"), (dict(positions=0), "ARG"),
    (dict(t=0), "DTYPE"), (dict(x=A + 1), "ALIGN"), (dict(y=B + 1), "ALIGN"), (dict(gamma=D + 2), "ALIGN"),
    (dict(turns=S1 + 4), "ALIGN"), (dict(positions=S2 + 4), "ALIGN"), (dict(t=2, x=A + 2), "ALIGN"),
    (dict(dim=15), "GEOMETRY"), (dict(dim=514), "GEOMETRY"), (dict(rot=15), "GEOMETRY"), (dict(rot=18), "GEOMETRY"),
    (dict(rows=2 ** 31), "GEOMETRY"), (dict(heads=65537), "GEOMETRY"), (dict(x_row=2 ** 41), "GEOMETRY"),
    (dict(y=A), "OVERLAP"), (dict(y=A, y_row=96, x_row=97), "OVERLAP"), (dict(y=A + 2, y_row=96), "OVERLAP"),
    (dict(gamma=B), "OVERLAP"), (dict(turns=B + 8), "OVERLAP"), (dict(positions=B + 16), "OVERLAP"),
    (dict(two=dict(KEYS, y=B + 32)), "OVERLAP"), (dict(two=dict(KEYS, y=A + 2)), "OVERLAP"),
    (dict(y_row=96, two=dict(KEYS, y=B + 96)), "OVERLAP"),        # the packed rows' tail reaches into the next row
    (dict(rows=0), "OK"), (dict(heads=0, x=0, y=0), "OK"), (dict(dim=0, rot=0), "OK"),
])
def test_heads_refusals(hm, kw, status):
    _is(hm, _heads(hm, **kw), status)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


@pytest.mark.parametrize("kw", [
    dict(), dict(y=A, y_row=96), dict(y=A, y_row=96, two=dict(KEYS, y=A + 128)),      # in place, packed
    dict(y_row=96, two=dict(KEYS, y=B + 128)), dict(y_row=16, y_head=48), dict(y_row=16, y_head=1000),
    dict(x_row=0, x_head=0), dict(heads=1, y_head=0), dict(rows=1, y_row=0), dict(gamma=0), dict(rot=0, turns=0, positions=0),
])
def test_layouts_that_pass_every_check(hm, kw):
    """Without a GPU a call that passes every check ends at the one for the device."""
    if not _no_gpu():
        pytest.skip("would launch on addresses that do not exist")
    assert _heads(hm, **kw) in (hm.HM_ERR_ARCH, hm.HM_ERR_CUDA)


def _elements(base, rows, row, heads, head, dim):
    """Element numbers of a matrix [rows][heads][dim], as a set."""
    return {base + r * row + h * head + e for r in range(rows) for h in range(heads) for e in range(dim)}


def test_no_overlap_is_missed(hm):
    """Small matrices at random places and strides: whenever an output shares an element with an input
    or another output, the call is refused; whenever a head's elements repeat, too."""
    if not _no_gpu():
        pytest.skip("would launch on addresses that do not exist")
    rng = np.random.default_rng(5)
    refused = passed = 0
    for _ in range(4000):
        rows, dim = int(rng.integers(1, 5)), 2 * int(rng.integers(1, 3))
        groups, sets = [], []
        for _ in range(int(rng.integers(1, 3))):
            heads = int(rng.integers(1, 4))
            m = [(int(rng.integers(0, 90)), int(rng.choice([0, dim, dim + 1, heads * dim, 3 * dim, 24, 40])),
                  int(rng.choice([0, dim, dim + 3, rows * dim, 12]))) for _ in range(2)]
            if rng.random() < 0.3:
                m[1] = m[0]  # in place
            groups.append((A + 2 * m[0][0], m[0][1], m[0][2], A + 2 * m[1][0], m[1][1], m[1][2], 0, heads))
            sets.append([_elements(b, rows, r, heads, h, dim) for b, r, h in m] + [rows * heads * dim, m[0] == m[1]])
        bad = False
        for i, (_, y, n, _) in enumerate(sets):
            bad |= len(y) < n
            for j, (x, z, _, in_place) in enumerate(sets):
                bad |= bool(y & x) and not (i == j and in_place)
                bad |= i != j and bool(y & z)
        got = _status(hm.head_norm_rope, hm.head_list(groups), hm.HM_BF16, rows, dim, 1e-6, None, 0)
        assert got != 0
        if bad:
            assert got in (hm.HM_ERR_OVERLAP, hm.HM_ERR_ARG), groups
        refused += bad
        passed += got not in (hm.HM_ERR_OVERLAP, hm.HM_ERR_ARG)
    assert refused > 500 and passed > 300


def test_number_of_groups(hm):
    g = hm.head_list([(A, 96, 16, B, 64, 16, 0, 0)] * 5)
    assert _status(hm.head_norm_rope, g, hm.HM_BF16, 3, 16, 1e-6, None, 0) == hm.HM_ERR_GEOMETRY
    assert _status(hm.head_norm_rope, hm.head_list([]), hm.HM_BF16, 3, 16, 1e-6, None, 0) == 0
    assert hm.lib().head_norm_rope(None, 1, hm.HM_BF16, 3, 16, 1e-6, None, None) == hm.HM_ERR_ARG


def _grad(hm, **kw):
    rot = _rotation(hm, kw)
    g = dict(dy=A, dy_row=64, dy_head=16, x=B, x_row=96, x_head=16, dx=X, dx_row=96, dx_head=16, gamma=D, dgamma=D + 4096,
             heads=4, acc=False)
    v = dict(t=hm.HM_BF16, rows=3, dim=16, eps=1e-6, ws=W, ws_bytes=1 << 20)
    two = kw.pop("two", None)
    for k, x in kw.items():
        (g if k in g else v)[k] = x
    groups = [tuple(g.values())] + ([tuple({**g, **two}.values())] if two else [])
    return _status(hm.head_norm_rope_backward, hm.head_grad_list(groups), v["t"], v["rows"], v["dim"], v["eps"], rot,
                   v["ws"], v["ws_bytes"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ARG"), (dict(dy=0), "ARG"), (dict(x=0), "ARG"), (dict(dx=0), "ARG"), (dict(gamma=0), "ARG"),
    (dict(heads=-1), "ARG"), (dict(dx_head=15), "ARG"), (dict(dx_row=63), "ARG"), (dict(dy_row=-1), "ARG"),
    (dict(layout=3), "ARG"), (dict(eps=-1.0), "ARG"), (dict(t=0), "DTYPE"), (dict(dy=A + 1), "ALIGN"),
    (dict(x=B + 1), "ALIGN"), (dict(dx=X + 1), "ALIGN"), (dict(dgamma=D + 4097), "ALIGN"), (dict(ws=W + 8), "ALIGN"),
    (dict(dim=514), "GEOMETRY"), (dict(rot=18), "GEOMETRY"), (dict(heads=65537), "GEOMETRY"),
    (dict(dx=A), "OVERLAP"), (dict(dx=B + 2), "OVERLAP"), (dict(dgamma=D), "OVERLAP"), (dict(dgamma=X), "OVERLAP"),
    (dict(dgamma=A), "OVERLAP"), (dict(dgamma=S1), "OVERLAP"), (dict(ws=A), "OVERLAP"), (dict(ws=X), "OVERLAP"),
    (dict(ws=S2), "OVERLAP"), (dict(ws=D), "OVERLAP"), (dict(dx=D), "OVERLAP"),
    (dict(two=dict(dy=Y, x=B + 128, dx=X + 128, heads=2)), "OVERLAP"),   # one dgamma for both
    (dict(heads=0, dgamma=0), "OK"), (dict(rows=0, dgamma=0), "OK"), (dict(dim=0, rot=0), "OK"),
])
def test_heads_gradient_refusals(hm, kw, status):
    _is(hm, _grad(hm, **kw), status)


def test_heads_gradient_workspace(hm):
    one = (A, 64, 16, B, 96, 16, X, 96, 16, D, D + 4096, 4, False)
    none = one[:10] + (0,) + one[11:]
    assert hm.head_norm_rope_backward_workspace(hm.head_grad_list([none]), 1000, 16) == 0
    assert hm.head_norm_rope_backward_workspace(hm.head_grad_list([one]), 0, 16) == 0
    assert hm.head_norm_rope_backward_workspace(hm.head_grad_list([one]), 1, 16) == 64
    assert hm.head_norm_rope_backward_workspace(hm.head_grad_list([one, none]), 1000, 16) % 64 == 0
    assert _status(hm.head_norm_rope_backward_workspace, hm.head_grad_list([one]), 5, 15) == hm.HM_ERR_GEOMETRY
    assert _status(hm.head_norm_rope_backward_workspace, hm.head_grad_list([one]), -1, 16) == hm.HM_ERR_ARG


@pytest.mark.parametrize("rot,theta,scaling,kw", [
    (2, 1e4, "unscaled", {}), (128, 1e4, "unscaled", {}), (24, 5e5, "linear", dict(factor=8.0)),
    (64, 1e4, "base", dict(factor=4.0)), (128, 1e6, "yarn", dict(factor=16.0, trained=4096.0)),
    (64, 1e4, "yarn", dict(factor=32.0, trained=8192.0, beta_fast=16.0, beta_slow=2.0)), (512, 1e4, "yarn", dict(factor=1.0, trained=1.0)),
])
def test_rope_turns(hm, rot, theta, scaling, kw):
    """Fixed point of freq / (2 pi): a few roundings in double precision (2^-48 is ample), then to
    the nearest 2^-64 turn, so off by at most 2^-65 turn = 2 pi 2^-65 = pi 2^-64 radians."""
    turns, scale = hm.rope_turns(rot, theta, ["unscaled", "linear", "base", "yarn"].index(scaling), **kw)
    f, s = OL.frequencies(rot, theta, scaling, **kw)
    assert len(turns) == rot // 2 and all(0 < t < 2 ** 62 for t in turns)
    got = np.array([t / 2.0 ** 64 for t in turns]) * 2 * np.pi
    assert (np.abs(got - f) <= f * 2.0 ** -48 + np.pi * 2.0 ** -64).all()
    assert abs(scale - s) <= s * 2.0 ** -24


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=3), "GEOMETRY"), (dict(rot_dim=0), "GEOMETRY"), (dict(rot_dim=514), "GEOMETRY"), (dict(theta=1.0), "ARG"),
    (dict(theta=float("inf")), "ARG"), (dict(scaling=4), "ARG"), (dict(scaling=-1), "ARG"), (dict(scaling=1, factor=0.5), "ARG"),
    (dict(scaling=1, factor=float("nan")), "ARG"), (dict(rot_dim=2, scaling=2), "GEOMETRY"),
    (dict(scaling=3, trained=0.0), "ARG"), (dict(scaling=3, trained=4096.0, beta_fast=1.0), "ARG"),
    (dict(scaling=3, trained=4096.0, beta_slow=0.0), "ARG"), (dict(scaling=2, theta=1e300, factor=1e20, rot_dim=4), "ARG"),
])
def test_rope_turns_refusals(hm, kw, status):
    _is(hm, _status(lambda: hm.rope_turns(**{"rot_dim": 16, **kw})), status)
