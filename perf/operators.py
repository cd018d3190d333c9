"""The operators around the update phase, as cases to measure: the MXFP8
product that reads the requantized weights, the norm and the quantization that
feed it, the norm's gradient, and the clipping of the gradient the update takes.

`run` makes the calls a user of the library makes (`own` true) or computes the
same in elementary torch operations in 32 bits, rounded once (`own` false);
`exact` computes the definitions in 64 bits.

MXFP8 operands are E4M3 codes [rows][K] with one UE8M0 scale per block of 32
(or 128, the scale stored four times) along K, the scales in the 128 x 4 tiled
layout.  Codes and scales are returned as the values they stand for.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one new token through a 5120-wide projection: the weight is read once, nothing else counts
        dict(name="gemm 1 token", op="gemm", m=1, n=5120, k=5120, out="bf16", acc=False, block=32, pad=0),
        # a short ragged batch through an expert's matrix, scales for each block of 128
        dict(name="gemm 77 tokens", op="gemm", m=77, n=1408, k=2048, out="bf16", acc=False, block=128, pad=0),
        # the forward product of a Video-DiT MLP over a full training batch
        dict(name="gemm fc1", op="gemm", m=8192, n=20480, k=5120, out="bf16", acc=False, block=32, pad=0),
        # a weight gradient (packed QKV of the language-model layer) added to the fp32 main gradient
        dict(name="gemm wgrad", op="gemm", m=6144, n=4096, k=4096, out="f32", acc=True, block=32, pad=0),
        # the norm before a projection for one new token
        dict(name="norm 1 token", op="norm", rows=1, d=5120, dtype="bf16", res=True, block=32),
        # the norm before fc1 over a full training batch
        dict(name="norm batch", op="norm", rows=8192, d=5120, dtype="bf16", res=True, block=32),
        # the norm's gradient for a few rows of a narrow expert model, residual stream kept in fp32
        dict(name="norm grad few rows", op="norm_grad", rows=33, d=2048, dtype="f32", res=True),
        # the norm's gradient over a full training batch
        dict(name="norm grad batch", op="norm_grad", rows=8192, d=5120, dtype="bf16", res=True),
        # an odd batch of activations, both directions, the norm's factors applied on the way
        dict(name="quantize odd", op="quantize", rows=131, cols=1408, dtype="bf16", rowwise=True, transposed=True,
             factors=True, block=32, pad=0),
        # the gradient of a packed QKV projection's output: one pass gives the operands of both its products
        dict(name="quantize both", op="quantize", rows=8192, cols=15360, dtype="bf16", rowwise=True, transposed=True,
             factors=False, block=32, pad=0),
        # the gradients of one small layer: latency counts
        dict(name="clip tiny", op="clip", tensors=5, mean=40000, dtype="f32", place="new", clipped=True, spread=1),
        # the gradients of one language-model layer with its norms, ragged sizes
        dict(name="clip layer", op="clip", tensors=48, mean=4194304, dtype="f32", place="new", clipped=True, spread=2),
    ]


MOST_FLOPS = 2.0 * 8192 * 20480 * 5120


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "norm", "norm_grad", "quantize", "clip"])
    dtype = rng.choice(["bf16", "f32"])
    block = rng.choice([32, 128])
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 64, 20480), 32 * _log(rng, 2, 640)
            if 2.0 * m * n * k <= MOST_FLOPS:
                break
        acc = dtype == "f32" and rng.random() < 0.5
        return dict(op=op, m=m, n=n, k=k, out=dtype, acc=acc, block=block, pad=rng.choice([0, 0, 3, 24]))
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 8192), d=32 * _log(rng, 2, 160), dtype=dtype, res=rng.random() < 0.8,
                    block=block)
    if op == "norm_grad":
        return dict(op=op, rows=_log(rng, 1, 8192), d=32 * _log(rng, 2, 160), dtype=dtype, res=rng.random() < 0.8)
    if op == "quantize":
        way = rng.choice([(True, True), (False, True), (True, False)])
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 33, 15360), dtype=dtype, rowwise=way[0],
                    transposed=way[1], factors=rng.random() < 0.5, block=block, pad=rng.choice([0, 0, 5, 32]))
    tensors = _log(rng, 1, 192)
    return dict(op=op, tensors=tensors, mean=_log(rng, 500, 200000000 // tensors), dtype=dtype,
                place=rng.choice(["new", "in"]), clipped=rng.random() < 0.7, spread=rng.randrange(3, 1000))


# ---- sizes ------------------------------------------------------------------
def _up(x, k):
    return -(-x // k) * k


def _type(name):
    return BF16 if name == "bf16" else F32


def _bytes(name):
    return 2 if name == "bf16" else 4


def _clip_sizes(c):
    """The tensors' element counts (norm weights, odd biases and matrices among them) and where each begins."""
    r = np.random.default_rng(c["spread"])
    n = np.maximum(1, (c["mean"] * r.uniform(0.05, 1.95, c["tensors"])).astype(np.int64))
    n[1::3] = np.maximum(1, n[1::3] // 512)
    gap = r.integers(0, 8, c["tensors"])  # elements: some tensors begin off any vector's boundary
    at = np.concatenate([[0], np.cumsum(n + gap)[:-1]])
    return [int(x) for x in n], [int(x) for x in at]


def _scale_bytes(rows, k):
    return _up(rows, 128) * _up(k // 32, 4)


def work(case):
    c = case
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        out = _bytes(c["out"]) * m * n * (2 if c["acc"] else 1)
        return {"bytes": (m + n) * k * (1 + 1 / 32) + out, "flops": 2.0 * m * n * k}
    if c["op"] == "norm":
        e, n = _bytes(c["dtype"]), c["rows"] * c["d"]
        return {"bytes": n * (e * (3 if c["res"] else 2) + 1 + 1 / 32) + 4 * c["rows"] + 4 * c["d"], "flops": 8.0 * n}
    if c["op"] == "norm_grad":
        e, n = _bytes(c["dtype"]), c["rows"] * c["d"]
        return {"bytes": n * e * (4 if c["res"] else 3) + 4 * c["rows"] + 8 * c["d"], "flops": 12.0 * n}
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        each = c["rowwise"] + c["transposed"]
        more = 4 * (c["rows"] + c["cols"]) if c["factors"] else 0
        return {"bytes": n * (_bytes(c["dtype"]) + each * (1 + 1 / 32)) + more, "flops": 4.0 * n * each}
    n = sum(_clip_sizes(c)[0])
    writes = c["place"] == "new" or c["clipped"]
    return {"bytes": n * _bytes(c["dtype"]) * (2 if writes else 1), "flops": (3.0 if writes else 2.0) * n}


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
    full = torch.zeros(rows, nb * block, dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, nb, block)
    amax = full.abs().max(dim=2, keepdim=True)[0]
    floor_log2 = lambda v: torch.frexp(v)[1].to(torch.float64) - 1.0  # noqa: E731  (log2 may round a power of two down)
    e = torch.where(amax > 0, floor_log2(amax) - 8, -127.0).clamp(-127, 127)
    y = full * torch.exp2(-e)
    step = torch.exp2(floor_log2(y.abs().clamp(min=2.0 ** -6)) - 3)
    y = (torch.round(y / step) * step).clamp(-448, 448).view(rows, -1)[:, :k]
    return y, torch.exp2(e[:, :, 0]).repeat_interleave(block // 32, dim=1)[:, :k // 32]


def _exact_tile(s):
    """Scale values laid out as _tile lays out bytes; the padding's zero byte stands for 2^-127."""
    rows, kb = s.shape
    out = torch.full((_up(rows, 128) // 128, _up(kb, 4) // 4, 32, 4, 4), 2.0 ** -127, dtype=torch.float64,
                     device=s.device)
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


def _operand(g, rows, k, block, weight):
    x = _normal(g, rows, k, std=0.02) if weight else _activations(g, rows, k, F32)
    q, s = _quantize(x, block)
    return q.contiguous(), _tile(s)


def _empty8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=c)
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        st["a"], st["sa"] = _operand(g, m, k, c["block"], False)
        st["b"], st["sb"] = _operand(g, n, k, c["block"], not c["acc"])
        d = torch.zeros(m, n + c["pad"], dtype=_type(c["out"]), device=DEV)
        if c["acc"]:
            d.copy_(_normal(g, m, n + c["pad"]))
        st["d"] = d
    elif c["op"] == "norm":
        rows, d, dt = c["rows"], c["d"], _type(c["dtype"])
        st["x"] = _activations(g, rows, d, dt)
        st["res"] = _activations(g, rows, d, dt) if c["res"] else None
        st["gamma"] = 1.0 + _normal(g, d, std=0.1)
        st["h"] = torch.empty(rows, d, dtype=dt, device=DEV)
        st["rstd"] = torch.empty(rows, dtype=F32, device=DEV)
        st["q"], st["s"] = _empty8(rows, d), _empty8(_scale_bytes(rows, d))
    elif c["op"] == "norm_grad":
        rows, d, dt = c["rows"], c["d"], _type(c["dtype"])
        st["dy"] = _normal(g, rows, d, std=1e-3).to(dt)
        st["dres"] = _normal(g, rows, d, std=1e-3).to(dt) if c["res"] else None
        st["h"] = _activations(g, rows, d, dt)
        st["gamma"] = 1.0 + _normal(g, d, std=0.1)
        st["rstd"] = torch.rsqrt(st["h"].to(F32).square().mean(dim=1) + EPS)
        st["dx"] = torch.empty(rows, d, dtype=dt, device=DEV)
        st["dgamma"] = torch.empty(d, dtype=F32, device=DEV)
    elif c["op"] == "quantize":
        rows, cols = c["rows"], c["cols"]
        st["x"] = _activations(g, rows, cols + c["pad"], _type(c["dtype"]))
        st["row"] = torch.exp(_normal(g, rows, std=0.3)) if c["factors"] else None
        st["col"] = 1.0 + _normal(g, cols, std=0.1) if c["factors"] else None
        if c["rowwise"]:
            st["q"], st["s"] = _empty8(rows, _up(cols, 32)), _empty8(_scale_bytes(rows, _up(cols, 32)))
        if c["transposed"]:
            st["qt"], st["st"] = _empty8(cols, _up(rows, 32)), _empty8(_scale_bytes(cols, _up(rows, 32)))
    else:
        n, at = _clip_sizes(c)
        flat = torch.zeros(at[-1] + n[-1], dtype=_type(c["dtype"]), device=DEV)
        flat.copy_(_normal(g, flat.numel(), std=1e-3))
        st["g"] = flat
        st["out"] = torch.zeros_like(flat) if c["place"] == "new" else flat
        st["parts"] = [(flat[a:a + k], st["out"][a:a + k]) for a, k in zip(at, n)]
        # the norm is about 1e-3 sqrt(elements)
        st["max_norm"] = 1e-3 * math.sqrt(sum(n)) * (0.3 if c["clipped"] else 3.0)
        st["stats"] = torch.zeros(2, dtype=F32, device=DEV)
    return st


# ---- one pass -------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _codes(q):
    return q.view(torch.float8_e4m3fn)


def _scales(s):
    return s.view(torch.float8_e8m0fnu)


def _plain_gemm(st):
    c = st["case"]
    a = _value(st["a"], _untile(st["sa"], c["m"], c["k"] // 32))
    b = _value(st["b"], _untile(st["sb"], c["n"], c["k"] // 32))
    d = st["d"][:, :c["n"]]
    r = a @ b.t()
    d.copy_(d + r if c["acc"] else r)
    return d


def _plain_norm(st):
    c = st["case"]
    h = st["x"].to(F32)
    if c["res"]:
        h = h + st["res"].to(F32)
    st["h"].copy_(h)
    h = st["h"].to(F32)  # the norm is of the stored residual stream
    rstd = 1.0 / torch.sqrt(h.square().mean(dim=1) + EPS)
    q, s = _quantize(h * rstd[:, None] * st["gamma"], c["block"])
    return {"h": st["h"], "rstd": rstd, "q": q, "s": _scales(_tile(s))}


def _plain_norm_grad(st):
    c = st["case"]
    xhat = st["h"].to(F32) * st["rstd"][:, None]
    dy = st["dy"].to(F32)
    t = dy * st["gamma"]
    dx = st["rstd"][:, None] * (t - xhat * (t * xhat).mean(dim=1, keepdim=True))
    if c["res"]:
        dx = dx + st["dres"].to(F32)
    return {"dx": dx.to(st["dx"].dtype), "dgamma": (dy * xhat).sum(dim=0)}


def _plain_quantize(st):
    c = st["case"]
    rows, cols = c["rows"], c["cols"]
    x = st["x"][:, :cols].to(F32)
    if c["factors"]:
        x = x * st["row"][:, None] * st["col"]
    out = {}
    if c["rowwise"]:
        q, s = _quantize(torch.nn.functional.pad(x, (0, _up(cols, 32) - cols)), c["block"])
        out["q"], out["s"] = q, _scales(_tile(s))
    if c["transposed"]:
        q, s = _quantize(torch.nn.functional.pad(x.t(), (0, _up(rows, 32) - rows)).contiguous(), c["block"])
        out["qt"], out["st"] = q, _scales(_tile(s))
    return out


def _plain_clip(st):
    norm = torch.sqrt(torch.stack([g.to(F32).square().sum() for g, _ in st["parts"]]).sum())
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(g.to(F32) * coef) for g, o in st["parts"]]
    return {"out": st["out"], "stats": torch.stack([norm, coef])}


_plain = dict(gemm=_plain_gemm, norm=_plain_norm, norm_grad=_plain_norm_grad, quantize=_plain_quantize,
              clip=_plain_clip)


def _abi():
    from head_muon_mxfp8_gb300 import abi
    return abi


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _dtype(abi, t):
    return abi.HM_BF16 if t.dtype == BF16 else abi.HM_F32


def _own_gemm(st):
    abi, c, d = _abi(), st["case"], st["d"]
    abi.mxfp8_gemm(_ptr(st["a"]), c["k"], _ptr(st["sa"]), _ptr(st["b"]), c["k"], _ptr(st["sb"]), c["m"], c["n"],
                   c["k"], _ptr(d), d.shape[1], _dtype(abi, d), c["acc"], _stream())
    return d[:, :c["n"]]


def _own_norm(st):
    abi, c = _abi(), st["case"]
    abi.rmsnorm_mxfp8(_ptr(st["x"]), c["d"], _ptr(st["res"]), _ptr(st["h"]), c["d"], _dtype(abi, st["x"]),
                      c["rows"], c["d"], _ptr(st["gamma"]), EPS, c["block"], _ptr(st["rstd"]), _ptr(st["q"]),
                      _ptr(st["s"]), _stream())
    return {"h": st["h"], "rstd": st["rstd"], "q": _codes(st["q"]), "s": _scales(st["s"])}


def _own_norm_grad(st):
    abi, c = _abi(), st["case"]
    if "ws" not in st:
        st["ws"] = _empty8(abi.rmsnorm_backward_workspace(c["rows"], c["d"]))
    abi.rmsnorm_backward(_ptr(st["dy"]), c["d"], _ptr(st["dres"]), _ptr(st["h"]), _ptr(st["dx"]), c["d"],
                         _dtype(abi, st["h"]), c["rows"], c["d"], _ptr(st["gamma"]), _ptr(st["rstd"]),
                         _ptr(st["dgamma"]), False, _ptr(st["ws"]), st["ws"].numel(), _stream())
    return {"dx": st["dx"], "dgamma": st["dgamma"]}


def _own_quantize(st):
    abi, c, x = _abi(), st["case"], st["x"]
    q, s, qt, s_t = (st.get(k) for k in ("q", "s", "qt", "st"))
    abi.mxfp8_quantize(_ptr(x), _dtype(abi, x), c["rows"], c["cols"], x.shape[1], _ptr(st["row"]), _ptr(st["col"]),
                       c["block"], _ptr(q), q.shape[1] if q is not None else 0, _ptr(s), _ptr(qt),
                       qt.shape[1] if qt is not None else 0, _ptr(s_t), _stream())
    out = {}
    if c["rowwise"]:
        out["q"], out["s"] = _codes(q), _scales(s)
    if c["transposed"]:
        out["qt"], out["st"] = _codes(qt), _scales(s_t)
    return out


def _own_clip(st):
    abi = _abi()
    if "list" not in st:
        st["list"] = abi.grad_list([(_ptr(g), _ptr(o), g.numel(), _dtype(abi, g)) for g, o in st["parts"]])
        st["ws"] = _empty8(abi.grad_norm_clip_workspace(st["list"]))
    abi.grad_norm_clip(st["list"], st["max_norm"], 1e-6, _ptr(st["stats"]), _ptr(st["ws"]), st["ws"].numel(),
                       _stream())
    return {"out": st["out"], "stats": st["stats"]}


_own = dict(gemm=_own_gemm, norm=_own_norm, norm_grad=_own_norm_grad, quantize=_own_quantize, clip=_own_clip)


# ---- the definitions in 64 bits --------------------------------------------------
def exact(case, seed):
    c, st = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "gemm":
        def operand(q, tiled, rows):
            kb = c["k"] // 32
            r = torch.arange(rows, device=DEV)[:, None]
            b = torch.arange(kb, device=DEV)[None, :]
            at = ((r // 128) * (_up(kb, 4) // 4) + b // 4) * 512 + (r % 32) * 16 + r % 128 // 32 * 4 + b % 4
            s = torch.exp2(tiled[at].to(f64) - 127.0)
            return (q.to(f64).view(rows, kb, 32) * s[:, :, None]).view(rows, c["k"])
        d = operand(st["a"], st["sa"], c["m"]) @ operand(st["b"], st["sb"], c["n"]).t()
        return d + st["d"][:, :c["n"]].to(f64) if c["acc"] else d
    if c["op"] == "norm":
        h = st["x"].to(f64) + (st["res"].to(f64) if c["res"] else 0.0)
        stored = h.to(_type(c["dtype"])).to(f64)
        rstd = (stored.square().sum(dim=1) / c["d"] + EPS) ** -0.5
        q, s = _exact_quantize(stored * rstd[:, None] * st["gamma"].to(f64), c["block"])
        return {"h": h, "rstd": rstd, "q": q, "s": _exact_tile(s)}
    if c["op"] == "norm_grad":
        # dL/dh of y = gamma h / sqrt(mean(h^2) + eps), rstd as given
        r, h, dy = st["rstd"].to(f64)[:, None], st["h"].to(f64), st["dy"].to(f64)
        t = dy * st["gamma"].to(f64)
        dx = r * t - r ** 3 * h * (t * h).sum(dim=1, keepdim=True) / c["d"]
        return {"dx": dx + (st["dres"].to(f64) if c["res"] else 0.0), "dgamma": (dy * h * r).sum(dim=0)}
    if c["op"] == "quantize":
        rows, cols = c["rows"], c["cols"]
        x = st["x"][:, :cols].to(f64)
        if c["factors"]:
            x = x * st["row"].to(f64)[:, None] * st["col"].to(f64)[None, :]
        out = {}
        if c["rowwise"]:
            wide = torch.zeros(rows, _up(cols, 32), dtype=f64, device=DEV)
            wide[:, :cols] = x
            q, s = _exact_quantize(wide, c["block"])
            out["q"], out["s"] = q, _exact_tile(s)
        if c["transposed"]:
            tall = torch.zeros(cols, _up(rows, 32), dtype=f64, device=DEV)
            tall[:, :rows] = x.t()
            q, s = _exact_quantize(tall, c["block"])
            out["qt"], out["st"] = q, _exact_tile(s)
        return out
    flat = st["g"].to(f64)
    out = st["out"].to(f64).clone()
    n, at = _clip_sizes(c)
    norm = math.sqrt(sum(float(flat[a:a + k].square().sum()) for a, k in zip(at, n)))
    coef = min(1.0, st["max_norm"] / (norm + 1e-6))
    for a, k in zip(at, n):
        out[a:a + k] = flat[a:a + k] * coef
    return {"out": out, "stats": torch.tensor([norm, coef], dtype=f64, device=DEV)}
