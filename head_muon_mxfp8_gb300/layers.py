"""The layers around the update whose matrices its units are cut from: the packed QKV
projection, whose heads are units of their own, and the MLP (fc1 and fc2, or gate, up
and down), on MXFP8 operands.

    qkv = NormQkv(tokens=4096, d_in=4096, q_heads=32, kv_heads=8, head_dim=128)
    q, k, v, h = qkv.forward(x, res, positions)        # heads normed and turned
    dx, dgamma = qkv.backward(dq, dk, dv, dres)

    mlp = NormMlp(tokens=4096, d=4096, d_ff=14336, activation="silu", gated=True)
    y, h = mlp.forward(x, res)                         # h = x + res, y = h + MLP(norm(h))
    dx, dgamma = mlp.backward(dy)

    layer.step(muon_hparams, max_norm=1.0)             # clip, Muon update, requantize

Buffers are allocated once; every computation runs in libhm's kernels on the current
stream.  Gradients add up until the next step().  Biases, gammas and their
gradients are the caller's to update (adamw_update_flat, before the next backward
pass).  Citations: SS-HSDP section 3.1 (EG1: main weight, runtime weight and
scales, per-head units of a packed QKV projection) and section 3.4 (the update's
place in a step)."""
from __future__ import annotations

from typing import List, Optional, Tuple

import torch

from . import _abi as abi
from .linear import MxBuffer, NormLinear, _need, _on_its_device, _ptr, _stream
from .session import MuonSession

ACTIVATIONS = {"none": abi.HM_ACT_NONE, "relu": abi.HM_ACT_RELU, "gelu": abi.HM_ACT_GELU,
               "gelu_tanh": abi.HM_ACT_GELU_TANH, "silu": abi.HM_ACT_SILU}
SCALINGS = {"unscaled": abi.HM_ROPE_UNSCALED, "linear": abi.HM_ROPE_LINEAR, "base": abi.HM_ROPE_BASE,
            "yarn": abi.HM_ROPE_YARN}


def _need_heads(name: str, t, shape: Tuple[int, int, int], device) -> None:
    """[tokens][heads][head_dim], the elements of a head next to each other, any strides else."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is expected, not {type(t).__name__}")
    if tuple(t.shape) != shape or t.dtype != torch.bfloat16 or t.device != device or t.stride(2) != 1:
        raise ValueError(f"{name}: a torch.bfloat16 tensor {list(shape)} on {device} with whole heads is expected, not "
                         f"{t.dtype} {list(t.shape)} with strides {list(t.stride())} on {t.device}")


def _rotation_table(rot_dim: int, theta: float, scaling: Optional[dict]):
    """abi.rope_turns of NormQkv's arguments; ([], 1.0) where nothing is rotated."""
    kw = dict(scaling or {"kind": "unscaled"})
    kind = kw.pop("kind", None)
    if kind not in SCALINGS:
        raise ValueError(f"scaling: a kind of {sorted(SCALINGS)} is expected, not {kind!r}")
    if kind != "unscaled" and "factor" not in kw:
        raise ValueError(f"scaling: {kind!r} needs a factor")
    if kind == "yarn" and kw.get("trained") is None:
        raise ValueError("scaling: 'yarn' needs `trained`, the positions that the model was trained on")
    return abi.rope_turns(rot_dim, theta, SCALINGS[kind], **kw) if rot_dim else ([], 1.0)


class NormQkv(NormLinear):
    """RMS norm, packed QKV projection (all query heads, then key heads, then value heads; a
    head is an update unit), norm of each query and key head and its rotation by position.
    rot_dim: the rotated part of a head (all of it by default); pairs: adjacent elements
    instead of halves; scaling: {"kind": "yarn", "factor": 16.0, "trained": 4096.0} and what else
    abi.rope_turns takes (ValueError where its kind, factor or YaRN's trained length is missing)."""

    def __init__(self, tokens: int, d_in: int, q_heads: int, kv_heads: int, head_dim: int, rot_dim: Optional[int] = None,
                 pairs: bool = False, theta: float = 10000.0, scaling: Optional[dict] = None, head_norm: bool = True,
                 eps: float = 1e-5, block: int = 32, device="cuda"):
        self.q_heads, self.kv_heads, self.head_dim, self.head_norm = q_heads, kv_heads, head_dim, head_norm
        rot_dim = head_dim if rot_dim is None else rot_dim
        if rot_dim > head_dim:
            raise ValueError(f"rot_dim: at most head_dim ({head_dim}) is expected, not {rot_dim}")
        turns, scale = _rotation_table(rot_dim, theta, scaling) if rot_dim or scaling else ([], 1.0)
        super().__init__(tokens, d_in, (q_heads + 2 * kv_heads) * head_dim, eps, block, device)
        self._rot = (scale, rot_dim, abi.HM_ROPE_PAIRS if pairs else abi.HM_ROPE_HALF)
        dev, f32 = self.device, dict(dtype=torch.float32, device=self.device)
        self._turns = torch.tensor(turns, dtype=torch.int64, device=dev)
        self.q = torch.empty(tokens, q_heads, head_dim, dtype=torch.bfloat16, device=dev)
        self.k = torch.empty(tokens, kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
        self.q_gamma, self.k_gamma = torch.ones(head_dim, **f32), torch.ones(head_dim, **f32)
        self.dq_gamma, self.dk_gamma = torch.zeros(head_dim, **f32), torch.zeros(head_dim, **f32)
        self._dy = torch.empty(tokens, self.d_out, dtype=torch.bfloat16, device=dev)
        self._positions = None   # of the forward pass
        self._head_ws = None
        if head_norm:
            self._clip += [(_ptr(t), _ptr(t), head_dim, abi.HM_F32) for t in (self.dq_gamma, self.dk_gamma)]

    def _units(self, d_out: int, d_in: int):
        dim = self.head_dim
        return [(i * dim * d_in, dim, d_in) for i in range(d_out // dim)]

    def _parts(self, packed: torch.Tensor):
        """Query, key and value heads of a packed [tokens][d_out]."""
        x = packed.view(self.tokens, -1, self.head_dim)
        a, b = self.q_heads, self.q_heads + self.kv_heads
        return x[:, :a], x[:, a:b], x[:, b:]

    def _gammas(self):
        return (self.q_gamma, self.k_gamma) if self.head_norm else (None, None)

    def _rotation(self):
        scale, rot_dim, layout = self._rot
        return abi.hm_rotation(_ptr(self._turns), _ptr(self._positions), scale, rot_dim, layout)

    @_on_its_device
    def forward(self, x: torch.Tensor, res: Optional[torch.Tensor], positions: torch.Tensor):
        """x, res: bf16 [tokens][d_in], positions: int64 [tokens] -> (q, k, v, h = x + res), q, k
        and v [tokens][heads][head_dim].  positions is read by the backward pass too."""
        _need("positions", positions, (self.tokens,), torch.int64, self.gamma.device)
        y, h = super().forward(x, res)
        self._positions = positions
        xq, xk, v = self._parts(y)
        groups = abi.head_list([(_ptr(a), *a.stride()[:2], _ptr(b), *b.stride()[:2], _ptr(g), a.shape[1])
                                for a, b, g in zip((xq, xk), (self.q, self.k), self._gammas())])
        abi.head_norm_rope(groups, abi.HM_BF16, self.tokens, self.head_dim, self.eps, self._rotation(), _stream())
        return self.q, self.k, v, h

    @_on_its_device
    def backward(self, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, dres: Optional[torch.Tensor] = None):
        """Gradients of q, k, v, bf16 [tokens][heads][head_dim] with whole heads, any strides else
        -> (dx, dgamma).  Adds dW to self.g and the gammas' gradients to self.dgamma, dq_gamma
        and dk_gamma."""
        dev = self.gamma.device
        for name, t, heads in (("dq", dq, self.q_heads), ("dk", dk, self.kv_heads), ("dv", dv, self.kv_heads)):
            _need_heads(name, t, (self.tokens, heads, self.head_dim), dev)
        if dres is not None:
            _need("dres", dres, (self.tokens, self.d_in), torch.bfloat16, dev)
        if self._positions is None:
            raise ValueError("backward: there was no forward pass")
        xq, xk, _ = self._parts(self.y)
        oq, ok, ov = self._parts(self._dy)
        dgammas = (self.dq_gamma, self.dk_gamma) if self.head_norm else (None, None)
        groups = abi.head_grad_list([(_ptr(t), *t.stride()[:2], _ptr(a), *a.stride()[:2], _ptr(o), *o.stride()[:2], _ptr(g),
                                      _ptr(dg), a.shape[1], self._summed)
                                     for t, a, o, g, dg in zip((dq, dk), (xq, xk), (oq, ok), self._gammas(), dgammas)])
        if self._head_ws is None:
            need = abi.head_norm_rope_backward_workspace(groups, self.tokens, self.head_dim)
            self._head_ws = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
        abi.head_norm_rope_backward(groups, abi.HM_BF16, self.tokens, self.head_dim, self.eps, self._rotation(),
                                    _ptr(self._head_ws), self._head_ws.numel(), _stream())
        ov.copy_(dv)
        return super().backward(self._dy, dres)


class _Weight:
    """A matrix [rows][cols] of the session: main weight and gradient, runtime codes, and the
    operands of both its products."""

    def __init__(self, session: MuonSession, offset: int, rows: int, cols: int, dev):
        a, n = session.bases[0] + offset, rows * cols
        self.rows, self.cols = rows, cols
        self.w, self.g = session.w[a:a + n].view(rows, cols), session.g[a:a + n].view(rows, cols)
        self.q, self.s = session.q[a:a + n].view(rows, cols), session.s[a // 32:(a + n) // 32]
        self.s_tiled = torch.zeros(abi.mxfp8_tiled_scale_bytes(rows, cols), dtype=torch.uint8, device=dev)
        self.t = MxBuffer(cols, rows, dev)

    def load(self, w: torch.Tensor, name: str) -> None:
        if tuple(w.shape) != (self.rows, self.cols):
            raise ValueError(f"{name}: [{self.rows}, {self.cols}] is expected, not {list(w.shape)}")
        self.w.copy_(w)
        abi.mxfp8_requant_packed(_ptr(self.w), _ptr(self.q), _ptr(self.s), [(0, 0, 0, self.rows, self.cols)], _stream())
        self.operands()

    def operands(self) -> None:
        """After a requantization: tiled scales, and the transpose from the main weight."""
        abi.mxfp8_scale_relayout(_ptr(self.s), _ptr(self.s_tiled), [(0, 0, self.rows, self.cols // 32, 1)], _stream())
        abi.mxfp8_quantize(_ptr(self.w), abi.HM_F32, self.rows, self.cols, self.cols, 0, 0, 32, 0, 0, 0, _ptr(self.t.q),
                           self.t.k, _ptr(self.t.s), _stream())


class NormMlp:
    """RMS norm and an MLP with the residual stream's addition.  gated: two first matrices, gate
    and up, and act(gate) * up; else fc1 and act(fc1).  bias: of the first matrices and the
    last one."""
    _summed = False   # whether the small gradients hold a backward pass since they were cleared
    _passed = False   # whether the buffers hold a whole forward pass

    def __init__(self, tokens: int, d: int, d_ff: int, activation: str = "gelu_tanh", gated: bool = False, bias: bool = True,
                 eps: float = 1e-5, block: int = 32, device="cuda"):
        if d % 32 or d_ff % 32:
            raise ValueError("d and d_ff are multiples of 32 (MX blocks)")
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation: one of {sorted(ACTIVATIONS)} is expected, not {activation!r}")
        self.tokens, self.d, self.d_ff, self.eps, self.block = tokens, d, d_ff, eps, block
        self.act, self.gated, self.has_bias = ACTIVATIONS[activation], gated, bias
        self.device = torch.device(device)
        self.gamma = torch.ones(d, dtype=torch.float32, device=self.device)
        self._allocate()

    @_on_its_device
    def _allocate(self) -> None:
        dev, tokens, d, ff = self.device, self.tokens, self.d, self.d_ff
        firsts = 2 if self.gated else 1
        units = [(i * ff * d, ff, d) for i in range(firsts)] + [(firsts * ff * d, d, ff)]
        self.session = MuonSession((firsts + 1) * ff * d, units, so=1, sw=1, sg=1, device=dev)
        self.weights: List[_Weight] = [_Weight(self.session, o, r, c, dev) for o, r, c in units]
        f32, bf16 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.bfloat16, device=dev)
        sizes = [ff] * firsts + [d]
        self.biases = [torch.zeros(n, **f32) for n in sizes] if self.has_bias else [None] * len(sizes)
        self.dbiases = [torch.zeros(n, **f32) for n in sizes] if self.has_bias else [None] * len(sizes)
        self.dgamma = torch.zeros(d, **f32)
        self.h, self.y, self.dn, self.dx = (torch.empty(tokens, d, **bf16) for _ in range(4))
        self.rstd = torch.empty(tokens, **f32)
        self.z = [torch.empty(tokens, ff, **bf16) for _ in range(firsts)]   # sums before the activation: fc1, or gate and up
        self.dz = [torch.empty(tokens, ff, **bf16) for _ in range(firsts)]
        self.a = torch.empty(tokens, ff, **bf16)
        self.x8, self.xt8 = MxBuffer(tokens, d, dev), MxBuffer(d, tokens, dev)          # norm(h)
        self.a8, self.at8 = MxBuffer(tokens, ff, dev), MxBuffer(ff, tokens, dev)
        self.dy8, self.dyt8 = MxBuffer(tokens, d, dev), MxBuffer(d, tokens, dev)
        self.dz8, self.dzt8 = MxBuffer(tokens, ff, dev), MxBuffer(ff, tokens, dev)
        need = max(abi.rmsnorm_backward_workspace(tokens, d), abi.mxfp8_quantize_bias_workspace(tokens, max(d, ff)), 16)
        self._ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self._clip = self.session.grad_list() + [(_ptr(t), _ptr(t), t.numel(), abi.HM_F32)
                                                 for t in [self.dgamma] + self.dbiases if t is not None]
        self.zero_grad()
        self.session.m.zero_()

    @_on_its_device
    def zero_grad(self) -> None:
        """Starts the gradients of a new step: clears the matrices'; the next backward pass overwrites
        the others (which stay readable until then) and later ones add to them."""
        self.session.g.zero_()
        self._summed = False

    @_on_its_device
    def load_weights(self, *ws: torch.Tensor) -> None:
        """fc1 and fc2, or gate, up and down: [d_ff][d] and, the last, [d][d_ff]."""
        if len(ws) != len(self.weights):
            raise ValueError(f"{len(self.weights)} matrices are expected, not {len(ws)}")
        for i, (w, t) in enumerate(zip(self.weights, ws)):
            w.load(t, f"matrix {i}")

    def _product(self, a: MxBuffer, b, b_scales, n: int, k: int, d: torch.Tensor, form: int, act: int, bias=None, first=None,
                 second=None, out2=None) -> None:
        """d [tokens][n] = epilogue of a [tokens][k] times codes b [n][k]."""
        e = abi.hm_epilogue(form, act, _ptr(bias), _ptr(first), n, _ptr(second), n, _ptr(out2), n)
        abi.mxfp8_gemm_epilogue(_ptr(a.q), a.k, _ptr(a.s), _ptr(b), k, _ptr(b_scales), self.tokens, n, k, _ptr(d), n,
                                abi.HM_BF16, e, _stream())

    def _quantize_gradient(self, x: torch.Tensor, q: MxBuffer, qt: MxBuffer, dbias: Optional[torch.Tensor]) -> None:
        """Both operands of a gradient's products, and the bias's gradient."""
        rows, cols = x.shape
        ops = (_ptr(q.q), q.k, _ptr(q.s), _ptr(qt.q), qt.k, _ptr(qt.s))
        if dbias is None:
            abi.mxfp8_quantize(_ptr(x), abi.HM_BF16, rows, cols, cols, 0, 0, self.block, *ops, _stream())
        else:
            abi.mxfp8_quantize_bias(_ptr(x), abi.HM_BF16, rows, cols, cols, self.block, *ops, _ptr(dbias), self._summed,
                                    _ptr(self._ws), self._ws.numel(), _stream())

    @_on_its_device
    def forward(self, x: torch.Tensor, res: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """x, res: bf16 [tokens][d], contiguous -> (y = h + MLP(norm(h)), h = x + res)."""
        for name, t in (("x", x), ("res", res)):
            if t is not None or name == "x":
                _need(name, t, (self.tokens, self.d), torch.bfloat16, self.gamma.device)
        self._passed = False
        st, d, ff = _stream(), self.d, self.d_ff
        abi.rmsnorm_mxfp8(_ptr(x), d, _ptr(res), _ptr(self.h), d, abi.HM_BF16, self.tokens, d, _ptr(self.gamma), self.eps,
                          self.block, _ptr(self.rstd), _ptr(self.x8.q), _ptr(self.x8.s), st)
        w, last = self.weights, self.weights[-1]
        if self.gated:
            self._product(self.x8, w[0].q, w[0].s_tiled, ff, d, self.z[0], abi.HM_EPI_FORWARD, abi.HM_ACT_NONE, self.biases[0])
            self._product(self.x8, w[1].q, w[1].s_tiled, ff, d, self.a, abi.HM_EPI_GATED, self.act, self.biases[1],
                          first=self.z[0], out2=self.z[1])
        else:
            self._product(self.x8, w[0].q, w[0].s_tiled, ff, d, self.a, abi.HM_EPI_FORWARD, self.act, self.biases[0],
                          out2=self.z[0])
        abi.mxfp8_quantize(_ptr(self.a), abi.HM_BF16, self.tokens, ff, ff, 0, 0, self.block, _ptr(self.a8.q), self.a8.k,
                           _ptr(self.a8.s), _ptr(self.at8.q), self.at8.k, _ptr(self.at8.s), st)
        self._product(self.a8, last.q, last.s_tiled, d, ff, self.y, abi.HM_EPI_FORWARD, abi.HM_ACT_NONE, self.biases[-1],
                      first=self.h)
        self._passed = True
        return self.y, self.h

    @_on_its_device
    def backward(self, dy: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """dy: bf16 [tokens][d], the gradient of y -> (dx, dgamma), dx of x and of res alike.  Adds
        to the matrices' gradients and, after the first pass of a step, to the others.  Of the
        forward pass before it (ValueError without one)."""
        _need("dy", dy, (self.tokens, self.d), torch.bfloat16, self.gamma.device)
        if not self._passed:
            raise ValueError("backward: there was no forward pass")
        st, d, ff, m = _stream(), self.d, self.d_ff, self.tokens
        last = self.weights[-1]
        self._quantize_gradient(dy, self.dy8, self.dyt8, self.dbiases[-1])
        # the gradient of what the activation took, straight from the second product's gradient
        if self.gated:
            self._product(self.dy8, last.t.q, last.t.s, ff, d, self.dz[1], abi.HM_EPI_GATED_GRADIENT, self.act,
                          first=self.z[0], second=self.z[1], out2=self.dz[0])
        else:
            self._product(self.dy8, last.t.q, last.t.s, ff, d, self.dz[0], abi.HM_EPI_GRADIENT, self.act, first=self.z[0])
        self._add_gradient(last, self.dyt8, self.at8)
        # norm(h)^T from h: the forward pass stored neither norm(h) nor its transpose
        abi.mxfp8_quantize(_ptr(self.h), abi.HM_BF16, m, d, d, _ptr(self.rstd), _ptr(self.gamma), self.block, 0, 0, 0,
                           _ptr(self.xt8.q), self.xt8.k, _ptr(self.xt8.s), st)
        for i, w in enumerate(self.weights[:-1]):
            self._quantize_gradient(self.dz[i], self.dz8, self.dzt8, self.dbiases[i])
            # gated: gate's part is rounded to bf16 before up's is added, half a step of it (2^-8) more than one
            # rounding of the sum, a fifteenth of what the operands' own rounding to E4M3 leaves (6 %)
            self._product(self.dz8, w.t.q, w.t.s, d, ff, self.dn, abi.HM_EPI_FORWARD, abi.HM_ACT_NONE,
                          first=self.dn if i else None)
            self._add_gradient(w, self.dzt8, self.xt8)
        abi.rmsnorm_backward(_ptr(self.dn), d, _ptr(dy), _ptr(self.h), _ptr(self.dx), d, abi.HM_BF16, m, d, _ptr(self.gamma),
                             _ptr(self.rstd), _ptr(self.dgamma), self._summed, _ptr(self._ws), self._ws.numel(), st)
        self._summed = True
        return self.dx, self.dgamma

    def _add_gradient(self, w: _Weight, dyt: MxBuffer, xt: MxBuffer) -> None:
        abi.mxfp8_gemm(_ptr(dyt.q), dyt.k, _ptr(dyt.s), _ptr(xt.q), xt.k, _ptr(xt.s), w.rows, w.cols, dyt.k, _ptr(w.g), w.cols,
                       abi.HM_F32, True, _stream())

    @_on_its_device
    def step(self, hp: "abi.hm_muon_hparams", max_norm: float = 1.0) -> torch.Tensor:
        """Clips all gradients by their global norm, runs the Muon update of the matrices (which
        requantizes them) and starts new gradients.  Returns (norm, coefficient) on the
        device."""
        stats = self.session.clip_grad_norm(max_norm, tensors=self._clip)
        self.session.run(hp, abi.HM_STAGE_ALL, torch.cuda.current_stream())
        for w in self.weights:
            w.operands()
        self.zero_grad()
        return stats

    def close(self) -> None:
        self.session.close()
