"""The operators of a layer's projections, as cases to measure: the MXFP8 product
with bias, activation, gate and residual in its epilogue and the same product's
gradient forms, the quantization that also sums a bias's gradient, and the norm of
query and key heads with the rotation by position, with its gradient.

`run` makes the calls a user of the library makes (`own` true) or computes the
same in elementary torch operations in 32 bits, rounded once (`own` false; the
rotation's angles in 64 bits); `exact` computes the definitions in 64 bits.

MXFP8 operands are E4M3 codes [rows][K] with one UE8M0 scale per block of 32 (or
128, the scale stored four times) along K, the scales in the 128 x 4 tiled layout.
Codes and scales are returned as the values they stand for.

A head's rotation turns pair i of its first `rot` elements by position * freq[i]:
elements (i, i + rot / 2) in the half layout, (2 i, 2 i + 1) in the interleaved one.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
TANH_A, TANH_B = math.sqrt(2.0 / math.pi), 0.044715


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # the up projection of the language-model layer for one new token, multiplied by its activated gate
        dict(name="gated 1 token", op="linear", form="gated", act="silu", m=1, n=14336, k=4096, out="bf16", bias=False,
             extra=True, keep=False, block=32, pad=0),
        # an expert's down projection of a ragged batch onto the fp32 residual stream
        dict(name="down ragged", op="linear", form="forward", act="none", m=777, n=2048, k=1408, out="f32", bias=True,
             extra=True, keep=False, block=32, pad=0),
        # the first projection of a Video-DiT MLP over a full training batch, its sum kept for the gradient
        dict(name="fc1 batch", op="linear", form="forward", act="gelu_tanh", m=8192, n=20480, k=5120, out="bf16",
             bias=True, extra=False, keep=True, block=32, pad=0),
        # the gradient of that projection's sum: the second projection's gradient product, times the activation's slope
        dict(name="fc1 gradient", op="linear", form="gradient", act="gelu_tanh", m=8192, n=20480, k=5120, out="bf16",
             bias=False, extra=True, keep=False, block=32, pad=0),
        # both gradients of an expert's gated pair for a ragged batch
        dict(name="gated gradient", op="linear", form="gated_gradient", act="silu", m=301, n=1408, k=2048, out="bf16",
             bias=False, extra=True, keep=True, block=128, pad=3),
        # an odd fp32 gradient: its operands of both products and the bias's gradient
        dict(name="bias odd", op="bias", rows=131, cols=1409, dtype="f32", rowwise=True, transposed=True, acc=True,
             block=128, pad=0),
        # the gradient of the Video-DiT MLP's first sum over a full batch
        dict(name="bias batch", op="bias", rows=8192, cols=20480, dtype="bf16", rowwise=True, transposed=True, acc=False,
             block=32, pad=0),
        # one new token of the language-model layer at a far position: 32 query and 8 key heads
        dict(name="heads 1 token", op="heads", rows=1, hq=32, hk=8, hv=8, dim=128, rot=128, layout="half", norm=True,
             scale=1.0, theta=1e6, stretch=1.0, far=1000000, dtype="bf16", place="rows"),
        # a full training batch of a Video-DiT layer: 40 query and 40 key heads out of the packed projection
        dict(name="heads batch", op="heads", rows=8192, hq=40, hk=40, hv=40, dim=128, rot=128, layout="half", norm=True,
             scale=1.0, theta=1e4, stretch=1.0, far=8192, dtype="bf16", place="heads"),
        # part of a narrow head, adjacent pairs, stretched positions, no norm
        dict(name="rotation partial", op="heads", rows=515, hq=12, hk=3, hv=3, dim=80, rot=24, layout="pairs", norm=False,
             scale=1.2, theta=1e4, stretch=8.0, far=100000, dtype="f32", place="rows"),
        # the gradient of a few rows' heads, fp32
        dict(name="heads gradient few", op="heads_grad", rows=33, hq=32, hk=8, hv=8, dim=128, rot=64, layout="pairs",
             norm=True, scale=1.0, theta=1e4, stretch=1.0, far=4096, dtype="f32", place="rows"),
        # the gradient of the full Video-DiT batch's heads
        dict(name="heads gradient batch", op="heads_grad", rows=8192, hq=40, hk=40, hv=40, dim=128, rot=128,
             layout="half", norm=True, scale=1.0, theta=1e4, stretch=1.0, far=8192, dtype="bf16", place="heads"),
    ]


MOST_FLOPS = 2.0 * 8192 * 20480 * 5120
MOST_HEADS = 8192 * 80 * 128  # elements of queries and keys


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "bias", "heads", "heads_grad"])
    dtype = rng.choice(["bf16", "f32"])
    block = rng.choice([32, 128])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 33, 20480), 32 * _log(rng, 2, 640)
            if 2.0 * m * n * k <= MOST_FLOPS:
                break
        form = rng.choice(["forward", "forward", "gated", "gradient", "gated_gradient"])
        grad = form in ("gradient", "gated_gradient")
        return dict(op=op, form=form, act=rng.choice(ACTS), m=m, n=n, k=k, out=dtype,
                    bias=not grad and rng.random() < 0.7,
                    extra=True if form != "forward" else rng.random() < 0.5,
                    keep=form == "gated_gradient" or (not grad and rng.random() < 0.5), block=block,
                    pad=rng.choice([0, 0, 3, 24]))
    if op == "bias":
        way = rng.choice([(True, True), (False, True), (True, False)])
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 33, 20480), dtype=dtype, rowwise=way[0],
                    transposed=way[1], acc=rng.random() < 0.5, block=block, pad=rng.choice([0, 0, 5, 32]))
    dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
    rot = rng.choice([dim, dim, dim // 2 // 2 * 2, dim // 4 // 2 * 2])
    hq, hk = rng.choice([(1, 1), (4, 4), (8, 1), (12, 3), (16, 16), (32, 8), (40, 40), (64, 8)])
    stretch = rng.choice([1.0, 1.0, 4.0, 32.0])
    most = min(16384, MOST_HEADS // ((hq + hk) * dim))
    return dict(op=op, rows=_log(rng, 1, most), hq=hq, hk=hk, hv=hk, dim=dim, rot=rot,
                layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.7,
                scale=1.0 if stretch == 1.0 else round(0.1 * math.log(stretch) + 1.0, 6),
                theta=rng.choice([1e4, 5e5, 1e6]), stretch=stretch, far=_log(rng, 64, 1000000), dtype=dtype,
                place=rng.choice(["rows", "heads"]))


# ---- sizes ------------------------------------------------------------------
def _up(x, k):
    return -(-x // k) * k


def _type(name):
    return BF16 if name == "bf16" else F32


def _bytes(name):
    return 2 if name == "bf16" else 4


def _scale_bytes(rows, k):
    return _up(rows, 128) * _up(k // 32, 4)


def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        # matrices of D's shape: D, what the epilogue reads and what else it writes
        reads = {"forward": int(c["extra"]), "gated": 1, "gradient": 1, "gated_gradient": 2}[c["form"]]
        each = _bytes(c["out"]) * m * n * (1 + reads + int(c["keep"]))
        return {"bytes": (m + n) * k * (1 + 1 / 32) + each + 4 * n * int(c["bias"]), "flops": 2.0 * m * n * k}
    if c["op"] == "bias":
        n = c["rows"] * c["cols"]
        each = c["rowwise"] + c["transposed"]
        return {"bytes": n * (_bytes(c["dtype"]) + each * (1 + 1 / 32)) + 4 * c["cols"] * (1 + c["acc"]),
                "flops": 5.0 * n}
    e = _bytes(c["dtype"])
    n = c["rows"] * (c["hq"] + c["hk"]) * c["dim"]
    small = 8 * c["rows"] + 4 * c["rot"] + (8 * c["dim"] if c["norm"] else 0)
    if c["op"] == "heads":
        return {"bytes": 2 * n * e + small, "flops": 8.0 * n}
    return {"bytes": n * e * (3 if c["norm"] else 2) + small + (8 * c["dim"] if c["norm"] else 0), "flops": 16.0 * n}


# ---- the format, in plain operations ------------------------------------------
def _tile(s):
    """Scales [rows][K / 32] in the 128 x 4 tiled layout: byte (r % 32) * 16 + (r / 32) * 4 + c of each tile."""
    rows, kb = s.shape
    full = torch.zeros(_up(rows, 128), _up(kb, 4), dtype=s.dtype, device=s.device)
    full[:rows, :kb] = s
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(t, rows, kb):
    cols = _up(kb, 4)
    full = t.view(-1, cols // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cols)
    return full[:rows, :kb]


def _quantize(x, block):
    """x [rows][K], K a multiple of 32, in 32 bits -> codes (E4M3) and the scales' bytes [rows][K / 32]."""
    rows, k = x.shape
    full = torch.nn.functional.pad(x, (0, _up(k, block) - k)) if k % block else x
    parts = full.view(rows, -1, block)
    amax = parts.abs().amax(dim=2)
    e = torch.where(amax == 0, -127, torch.frexp(amax)[1] - 9).clamp(-127, 127)
    q = torch.ldexp(parts, -e[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, -1)[:, :k]
    s = (e + 127).to(torch.uint8).repeat_interleave(block // 32, dim=1)[:, :k // 32]
    return q, s


def _value(q, s):
    """The 32-bit values of codes [rows][K] with scale bytes [rows][K / 32]."""
    x = q.to(F32).view(q.shape[0], -1, 32)
    return torch.ldexp(x, s.to(torch.int32)[:, :, None] - 127).view(q.shape)


def _exact_quantize(x, block):
    """The same from the format's definition, in 64 bits: the codes' and the scales' values."""
    rows, k = x.shape
    nb = -(-k // block)
    full = torch.zeros(rows, nb * block, dtype=F64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, nb, block)
    amax = full.abs().max(dim=2, keepdim=True)[0]
    floor_log2 = lambda v: torch.frexp(v)[1].to(F64) - 1.0  # noqa: E731  (log2 may round a power of two down)
    e = torch.where(amax > 0, floor_log2(amax) - 8, -127.0).clamp(-127, 127)
    y = full * torch.exp2(-e)
    step = torch.exp2(floor_log2(y.abs().clamp(min=2.0 ** -6)) - 3)
    y = (torch.round(y / step) * step).clamp(-448, 448).view(rows, -1)[:, :k]
    return y, torch.exp2(e[:, :, 0]).repeat_interleave(block // 32, dim=1)[:, :k // 32]


def _exact_tile(s):
    """Scale values laid out as _tile lays out bytes; the padding's zero byte stands for 2^-127."""
    rows, kb = s.shape
    out = torch.full((_up(rows, 128) // 128, _up(kb, 4) // 4, 32, 4, 4), 2.0 ** -127, dtype=F64, device=s.device)
    r, c = torch.meshgrid(torch.arange(rows, device=s.device), torch.arange(kb, device=s.device), indexing="ij")
    out[r // 128, c // 4, r % 32, r % 128 // 32, c % 4] = s
    return out.view(-1)


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=F32, device=DEV).normal_(0.0, std, generator=g)


def _activations(g, rows, cols, dtype):
    """Gaussian rows of different sizes, with a few channels much larger than the others."""
    x = _normal(g, rows, cols)
    x *= torch.exp(_normal(g, rows, 1, std=0.5))
    x *= torch.where(torch.rand(cols, device=DEV, generator=g) < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _operand(g, rows, k, block, kind):
    if kind == "weight":
        x = _normal(g, rows, k, std=k ** -0.5)
    elif kind == "gradient":
        x = _normal(g, rows, k, std=1e-3)
    else:
        x = _normal(g, rows, k) * torch.exp(_normal(g, rows, 1, std=0.5))
    q, s = _quantize(x, block)
    return q.contiguous(), _tile(s)


def _empty8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device=DEV)


def _matrix(g, c, std):
    """A matrix of D's shape and pitch."""
    return _normal(g, c["m"], c["n"] + c["pad"], std=std).to(_type(c["out"]))


def _frequencies(c):
    """Radians per position of each pair, in 64 bits, and the same as turns in units of 2^-64 turn."""
    freq = np.power(c["theta"], -2.0 * np.arange(c["rot"] // 2) / c["rot"]) / c["stretch"]
    turns = [int(round(f / (2.0 * math.pi) * 2.0 ** 64)) for f in freq]
    turns = np.array([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=np.int64)
    return torch.from_numpy(freq).to(DEV), torch.from_numpy(turns).to(DEV)


def _by_place(c, heads, fill):
    """[rows][heads][dim], stored in that order or head by head."""
    if c["place"] == "rows":
        return fill(c["rows"], heads, c["dim"])
    return fill(heads, c["rows"], c["dim"]).transpose(0, 1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=c)
    if c["op"] == "linear":
        m, n, k, form = c["m"], c["n"], c["k"], c["form"]
        grad = form in ("gradient", "gated_gradient")
        st["a"], st["sa"] = _operand(g, m, k, c["block"], "gradient" if grad else "activation")
        st["b"], st["sb"] = _operand(g, n, k, c["block"], "weight")
        st["bias"] = _normal(g, n, std=0.3) if c["bias"] else None
        # the residual stream; sums before an activation lie where the activation bends
        st["in"] = _matrix(g, c, 3.0 if form == "forward" else 1.5) if c["extra"] else None
        st["in2"] = _matrix(g, c, 1.0) if form == "gated_gradient" else None
        st["d"] = torch.zeros(m, n + c["pad"], dtype=_type(c["out"]), device=DEV)
        st["out2"] = torch.zeros_like(st["d"]) if c["keep"] else None
    elif c["op"] == "bias":
        rows, cols = c["rows"], c["cols"]
        st["x"] = (_activations(g, rows, cols + c["pad"], F32) * 1e-3).to(_type(c["dtype"]))
        st["before"] = _normal(g, cols, std=1e-2)  # of the micro-batches before
        st["db"] = torch.zeros(cols, dtype=F32, device=DEV)
        if c["rowwise"]:
            st["q"], st["s"] = _empty8(rows, _up(cols, 32)), _empty8(_scale_bytes(rows, _up(cols, 32)))
        if c["transposed"]:
            st["qt"], st["st"] = _empty8(cols, _up(rows, 32)), _empty8(_scale_bytes(cols, _up(rows, 32)))
    else:
        rows, dim, dt = c["rows"], c["dim"], _type(c["dtype"])
        heads = c["hq"] + c["hk"] + c["hv"]
        st["x"] = _activations(g, rows, heads * dim, dt).view(rows, heads, dim)
        # positions of packed sequences, the last one far out
        st["pos"] = torch.randint(0, c["far"], (rows,), device=DEV, generator=g)
        st["pos"][-1] = c["far"]
        st["freq"], st["turns"] = _frequencies(c)
        for name, n in (("q", c["hq"]), ("k", c["hk"])):
            st["g" + name] = 1.0 + _normal(g, dim, std=0.1) if c["norm"] else None
            if c["op"] == "heads":
                st[name] = _by_place(c, n, lambda *s: torch.zeros(*s, dtype=dt, device=DEV))
            else:
                st["d" + name] = _by_place(c, n, lambda *s: _normal(g, *s, std=1e-3).to(dt))
                st["dg" + name] = torch.zeros(dim, dtype=F32, device=DEV) if c["norm"] else None
        if c["op"] == "heads_grad":
            st["dx"] = torch.zeros_like(st["x"])
    return st


# ---- one pass -------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _codes(q):
    return q.view(torch.float8_e4m3fn)


def _scales(s):
    return s.view(torch.float8_e8m0fnu)


def _act(name, z):
    """The activation and its slope."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.clamp(z, min=0.0), (z > 0).to(z.dtype)
    if name == "gelu":
        phi = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(TANH_A * (z + TANH_B * z * z * z))
        return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * TANH_A * (1.0 + 3.0 * TANH_B * z * z)
    s = torch.sigmoid(z)
    return z * s, s + z * s * (1.0 - s)


def _linear_outputs(c, d, out2):
    return {"d": d, "out2": out2} if c["keep"] else {"d": d}


def _plain_linear(st):
    c = st["case"]
    n, dt = c["n"], _type(c["out"])
    a = _value(st["a"], _untile(st["sa"], c["m"], c["k"] // 32))
    b = _value(st["b"], _untile(st["sb"], n, c["k"] // 32))
    z = a @ b.t()
    if c["bias"]:
        z = z + st["bias"]
    x = st["in"][:, :n].to(F32) if c["extra"] else None
    out2 = None
    if c["form"] == "forward":
        out2, y = z, _act(c["act"], z)[0]
        y = y + x if c["extra"] else y
    elif c["form"] == "gated":
        out2, y = z, z * _act(c["act"], x)[0]
    elif c["form"] == "gradient":
        y = z * _act(c["act"], x)[1]
    else:
        value, slope = _act(c["act"], x)
        y, out2 = z * value, z * st["in2"][:, :n].to(F32) * slope
    return _linear_outputs(c, y.to(dt), out2.to(dt) if c["keep"] else None)


def _plain_bias(st):
    c = st["case"]
    rows, cols = c["rows"], c["cols"]
    x = st["x"][:, :cols].to(F32)
    out = {"db": x.sum(dim=0) + st["before"] if c["acc"] else x.sum(dim=0)}
    if c["rowwise"]:
        q, s = _quantize(torch.nn.functional.pad(x, (0, _up(cols, 32) - cols)), c["block"])
        out["q"], out["s"] = q, _scales(_tile(s))
    if c["transposed"]:
        q, s = _quantize(torch.nn.functional.pad(x.t(), (0, _up(rows, 32) - rows)).contiguous(), c["block"])
        out["qt"], out["st"] = q, _scales(_tile(s))
    return out


def _angles(st):
    """cos and sin [rows][1][rot / 2], angles in 64 bits, the scale applied."""
    c = st["case"]
    a = st["pos"].to(F64)[:, None] * st["freq"]
    return (torch.cos(a) * c["scale"])[:, None], (torch.sin(a) * c["scale"])[:, None]


def _rotate(c, v, cos, sin):
    """v [rows][heads][dim] rotated; -sin turns back."""
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = v[..., :rot // 2], v[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = v[..., 0:rot:2], v[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, v[..., rot:]], dim=-1)


def _heads_of(c, x):
    return (("q", x[:, :c["hq"]]), ("k", x[:, c["hq"]:c["hq"] + c["hk"]]))


def _plain_heads(st):
    c, out = st["case"], {}
    cos, sin = (t.to(F32) for t in _angles(st))
    for name, x in _heads_of(c, st["x"]):
        v = x.to(F32)
        if c["norm"]:
            v = v * (1.0 / torch.sqrt(v.square().mean(dim=-1, keepdim=True) + EPS)) * st["g" + name]
        st[name].copy_(_rotate(c, v, cos, sin))
        out[name] = st[name]
    return out


def _plain_heads_grad(st):
    c, out = st["case"], {"dx": st["dx"]}
    cos, sin = (t.to(F32) for t in _angles(st))
    for (name, x), (_, dx) in zip(_heads_of(c, st["x"]), _heads_of(c, st["dx"])):
        t = _rotate(c, st["d" + name].to(F32), cos, -sin)
        if c["norm"]:
            v = x.to(F32)
            r = 1.0 / torch.sqrt(v.square().mean(dim=-1, keepdim=True) + EPS)
            xhat = v * r
            out["dg" + name] = (t * xhat).sum(dim=(0, 1))
            t = t * st["g" + name]
            t = r * (t - xhat * (t * xhat).mean(dim=-1, keepdim=True))
        dx.copy_(t)
    return out


_plain = dict(linear=_plain_linear, bias=_plain_bias, heads=_plain_heads, heads_grad=_plain_heads_grad)


def _abi():
    from head_muon_mxfp8_gb300 import abi
    return abi


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _dtype(abi, t):
    return abi.HM_BF16 if t.dtype == BF16 else abi.HM_F32


def _own_linear(st):
    abi, c, d = _abi(), st["case"], st["d"]
    if "epilogue" not in st:
        ld = d.shape[1]
        st["epilogue"] = abi.hm_epilogue(getattr(abi, "HM_EPI_" + c["form"].upper()),
                                         getattr(abi, "HM_ACT_" + c["act"].upper()), _ptr(st["bias"]), _ptr(st["in"]), ld,
                                         _ptr(st["in2"]), ld, _ptr(st["out2"]), ld)
    abi.mxfp8_gemm_epilogue(_ptr(st["a"]), c["k"], _ptr(st["sa"]), _ptr(st["b"]), c["k"], _ptr(st["sb"]), c["m"], c["n"],
                            c["k"], _ptr(d), d.shape[1], _dtype(abi, d), st["epilogue"], _stream())
    n = c["n"]
    return _linear_outputs(c, d[:, :n], st["out2"][:, :n] if c["keep"] else None)


def _own_bias(st):
    abi, c, x = _abi(), st["case"], st["x"]
    if "ws" not in st:
        st["ws"] = _empty8(abi.mxfp8_quantize_bias_workspace(c["rows"], c["cols"]))
    if c["acc"]:
        st["db"].copy_(st["before"])
    q, s, qt, s_t = (st.get(k) for k in ("q", "s", "qt", "st"))
    abi.mxfp8_quantize_bias(_ptr(x), _dtype(abi, x), c["rows"], c["cols"], x.shape[1], c["block"], _ptr(q),
                            q.shape[1] if q is not None else 0, _ptr(s), _ptr(qt), qt.shape[1] if qt is not None else 0,
                            _ptr(s_t), _ptr(st["db"]), c["acc"], _ptr(st["ws"]), st["ws"].numel(), _stream())
    out = {"db": st["db"]}
    if c["rowwise"]:
        out["q"], out["s"] = _codes(q), _scales(s)
    if c["transposed"]:
        out["qt"], out["st"] = _codes(qt), _scales(s_t)
    return out


def _rotation(abi, st):
    c = st["case"]
    return abi.hm_rotation(_ptr(st["turns"]), _ptr(st["pos"]), c["scale"], c["rot"],
                           abi.HM_ROPE_HALF if c["layout"] == "half" else abi.HM_ROPE_PAIRS)


def _row_head(t):
    return t.stride(0), t.stride(1)


def _own_heads(st):
    abi, c = _abi(), st["case"]
    if "groups" not in st:
        st["groups"] = abi.head_list([(_ptr(x), *_row_head(x), _ptr(st[name]), *_row_head(st[name]), _ptr(st["g" + name]),
                                       x.shape[1]) for name, x in _heads_of(c, st["x"])])
        st["rotation"] = _rotation(abi, st)
    abi.head_norm_rope(st["groups"], _dtype(abi, st["x"]), c["rows"], c["dim"], EPS, st["rotation"], _stream())
    return {"q": st["q"], "k": st["k"]}


def _own_heads_grad(st):
    abi, c = _abi(), st["case"]
    if "groups" not in st:
        st["groups"] = abi.head_grad_list(
            [(_ptr(st["d" + name]), *_row_head(st["d" + name]), _ptr(x), *_row_head(x), _ptr(dx), *_row_head(dx),
              _ptr(st["g" + name]), _ptr(st["dg" + name]), x.shape[1], False)
             for (name, x), (_, dx) in zip(_heads_of(c, st["x"]), _heads_of(c, st["dx"]))])
        st["rotation"] = _rotation(abi, st)
        st["ws"] = _empty8(max(1, abi.head_norm_rope_backward_workspace(st["groups"], c["rows"], c["dim"])))
    abi.head_norm_rope_backward(st["groups"], _dtype(abi, st["x"]), c["rows"], c["dim"], EPS, st["rotation"],
                                _ptr(st["ws"]), st["ws"].numel(), _stream())
    out = {"dx": st["dx"]}
    if c["norm"]:
        out["dgq"], out["dgk"] = st["dgq"], st["dgk"]
    return out


_own = dict(linear=_own_linear, bias=_own_bias, heads=_own_heads, heads_grad=_own_heads_grad)


# ---- the definitions in 64 bits --------------------------------------------------
def _exact_act(name, z):
    """(f(z), f'(z)) of the activation f."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(F64)
        return z * on, on
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    # z / (1 + exp(-u)) with u = z, or u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
    u, du = (z, 1.0) if name == "silu" else (2 * TANH_A * (z + TANH_B * z ** 3), 2 * TANH_A * (1 + 3 * TANH_B * z ** 2))
    s = 1.0 / (1.0 + torch.exp(-u))
    return z * s, s + z * s * (1.0 - s) * du


def _exact_linear(c, st):
    def operand(q, tiled, rows):
        kb = c["k"] // 32
        r = torch.arange(rows, device=DEV)[:, None]
        b = torch.arange(kb, device=DEV)[None, :]
        at = ((r // 128) * (_up(kb, 4) // 4) + b // 4) * 512 + (r % 32) * 16 + r % 128 // 32 * 4 + b % 4
        s = torch.exp2(tiled[at].to(F64) - 127.0)
        return (q.to(F64).view(rows, kb, 32) * s[:, :, None]).view(rows, c["k"])
    n = c["n"]
    p = operand(st["a"], st["sa"], c["m"]) @ operand(st["b"], st["sb"], n).t()
    if c["bias"]:
        p += st["bias"].to(F64)
    x = st["in"][:, :n].to(F64) if c["extra"] else None
    if c["form"] == "forward":
        d = _exact_act(c["act"], p)[0] + (x if c["extra"] else 0.0)
        return _linear_outputs(c, d, p)
    f, slope = _exact_act(c["act"], x)
    if c["form"] == "gated":
        return _linear_outputs(c, p * f, p)
    if c["form"] == "gradient":
        return _linear_outputs(c, p * slope, None)
    return _linear_outputs(c, p * f, p * st["in2"][:, :n].to(F64) * slope)


def _exact_bias(c, st):
    rows, cols = c["rows"], c["cols"]
    x = st["x"][:, :cols].to(F64)
    out = {"db": x.sum(dim=0) + (st["before"].to(F64) if c["acc"] else 0.0)}
    if c["rowwise"]:
        wide = torch.zeros(rows, _up(cols, 32), dtype=F64, device=DEV)
        wide[:, :cols] = x
        q, s = _exact_quantize(wide, c["block"])
        out["q"], out["s"] = q, _exact_tile(s)
    if c["transposed"]:
        tall = torch.zeros(cols, _up(rows, 32), dtype=F64, device=DEV)
        tall[:, :rows] = x.t()
        q, s = _exact_quantize(tall, c["block"])
        out["qt"], out["st"] = q, _exact_tile(s)
    return out


def _exact_turn(c, st, v, back):
    """Pair i of each head as a complex number, times scale * exp(i angle) (back: its transpose)."""
    rot, h = c["rot"], c["rot"] // 2
    i = torch.arange(h, device=DEV)
    at, to = (i, i + h) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    angle = (st["pos"].to(F64)[:, None] * st["freq"])[:, None, :]
    z = torch.complex(v[..., at].contiguous(), v[..., to].contiguous())
    z = z * torch.polar(torch.full_like(angle, c["scale"]), -angle if back else angle)
    out = v.clone()
    out[..., at], out[..., to] = z.real, z.imag
    return out


def _exact_heads(c, st):
    out = {}
    for name, x in _heads_of(c, st["x"]):
        v = x.to(F64)
        if c["norm"]:
            v = v * (v.square().sum(dim=-1, keepdim=True) / c["dim"] + EPS) ** -0.5 * st["g" + name].to(F64)
        out[name] = _exact_turn(c, st, v, False)
    return out


def _exact_heads_grad(c, st):
    dx, out = st["dx"].to(F64), {}
    for (name, x), (_, part) in zip(_heads_of(c, st["x"]), _heads_of(c, dx)):
        t = _exact_turn(c, st, st["d" + name].to(F64), True)
        if c["norm"]:
            v = x.to(F64)
            r = (v.square().sum(dim=-1, keepdim=True) / c["dim"] + EPS) ** -0.5
            out["dg" + name] = (t * v * r).sum(dim=(0, 1))
            t = t * st["g" + name].to(F64)
            t = r * t - r ** 3 * v * (t * v).sum(dim=-1, keepdim=True) / c["dim"]
        part.copy_(t)
    return {"dx": dx, **out}


def exact(case, seed):
    return dict(linear=_exact_linear, bias=_exact_bias, heads=_exact_heads, heads_grad=_exact_heads_grad)[case["op"]](
        case, prepare(case, seed))
