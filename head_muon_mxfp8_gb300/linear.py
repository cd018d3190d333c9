"""An RMS norm and a linear layer on MXFP8 operands, around the update: the
runtime weight is what the Muon session's update requantizes, the weight
gradient lands in the session's main gradient.

    layer = NormLinear(tokens=4096, d_in=5120, d_out=15360)
    layer.load_weight(w)                       # fp32 main weight [d_out][d_in]
    y, h = layer.forward(x, res)               # h = x + res, y = norm(h) W^T
    dx, dgamma = layer.backward(dy, dres)      # dW and dgamma add up until the next step()
    layer.step(muon_hparams, max_norm=1.0)     # clip, Muon update, requantize

Buffers are allocated once; every computation runs in libhm's kernels on the
current stream.  One emulated rank: the weight is one contiguous matrix of the
session's roots.  Citations: SS-HSDP section 3.1 (EG1: main weight, runtime
weight and scales, main gradient) and section 3.4 (the update's place in a
step)."""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import _abi as abi
from .session import MuonSession


def _up(x: int, k: int) -> int:
    return -(-x // k) * k


class MxBuffer:
    """Codes [rows][k32] (k rounded up to 32) and tiled scales of one MXFP8 operand."""

    def __init__(self, rows: int, k: int, device):
        self.rows, self.k = rows, _up(k, 32)
        self.q = torch.zeros(rows, self.k, dtype=torch.uint8, device=device)
        self.s = torch.zeros(abi.mxfp8_tiled_scale_bytes(rows, self.k), dtype=torch.uint8, device=device)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _on_its_device(method):
    """Runs a layer's method with the layer's device current: its streams and launches."""
    @functools.wraps(method)
    def run(self, *args, **kw):
        with torch.cuda.device_of(self.gamma):
            return method(self, *args, **kw)
    return run


def _ptr(t: Optional[torch.Tensor]) -> int:
    return t.data_ptr() if t is not None else 0


def _need(name: str, t, shape: Tuple[int, int], dtype, device) -> None:
    """The kernels take addresses: t has to be what they will read there."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is expected, not {type(t).__name__}")
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor {list(shape)} on {device} is expected, not {t.dtype} "
                         f"{list(t.shape)} with strides {list(t.stride())} on {t.device}")


class NormLinear:
    _summed = False   # whether dgamma holds a backward pass since the gradients were cleared

    def __init__(self, tokens: int, d_in: int, d_out: int, eps: float = 1e-5, block: int = 32, device="cuda"):
        """Buffers for `tokens` rows on `device`, which need not be the current one."""
        if d_in % 32 or d_out % 32:
            raise ValueError("d_in and d_out are multiples of 32 (MX blocks)")
        self.tokens, self.d_in, self.d_out, self.eps, self.block = tokens, d_in, d_out, eps, block
        dev = self.device = torch.device(device)
        self.gamma = torch.ones(d_in, dtype=torch.float32, device=dev)
        self._allocate(tokens, d_in, d_out, dev)

    @_on_its_device
    def _allocate(self, tokens: int, d_in: int, d_out: int, dev) -> None:
        self.session = MuonSession(d_out * d_in, [(0, d_out, d_in)], so=1, sw=1, sg=1, device=dev)
        base, n = self.session.bases[0], d_out * d_in
        self.w = self.session.w[base:base + n].view(d_out, d_in)   # fp32 main weight
        self.g = self.session.g[base:base + n].view(d_out, d_in)   # fp32 main gradient
        self._q = self.session.q[base:base + n].view(d_out, d_in)  # runtime weight's codes
        self._s = self.session.s[base // 32:(base + n) // 32]      # its K-major scales
        self._s_tiled = torch.zeros(abi.mxfp8_tiled_scale_bytes(d_out, d_in), dtype=torch.uint8, device=dev)
        self.wt = MxBuffer(d_in, d_out, dev)                       # W^T, for the gradient of x
        self.dgamma = torch.zeros(d_in, dtype=torch.float32, device=dev)
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        self.h = torch.empty(tokens, d_in, **bf16)
        self.rstd = torch.empty(tokens, dtype=torch.float32, device=dev)
        self.y = torch.empty(tokens, d_out, **bf16)
        self.x8 = MxBuffer(tokens, d_in, dev)       # norm(h)
        self.xt8 = MxBuffer(d_in, tokens, dev)      # norm(h)^T
        self.dy8 = MxBuffer(tokens, d_out, dev)
        self.dyt8 = MxBuffer(d_out, tokens, dev)
        self.dn = torch.empty(tokens, d_in, **bf16)  # gradient of norm(h)
        self.dx = torch.empty(tokens, d_in, **bf16)
        self._ws = torch.empty(abi.rmsnorm_backward_workspace(tokens, d_in), dtype=torch.uint8, device=dev)
        self._clip = self.session.grad_list() + [(_ptr(self.dgamma), _ptr(self.dgamma), d_in, abi.HM_F32)]
        self.zero_grad()
        self.session.m.zero_()

    @_on_its_device
    def zero_grad(self) -> None:
        """Starts the gradients of a new step: clears dW; the next backward pass overwrites
        dgamma (which stays readable until then) and later ones add to it."""
        self.g.zero_()
        self._summed = False

    @_on_its_device
    def load_weight(self, w: torch.Tensor) -> None:
        """w [d_out][d_in], any floating type, layout and device (ValueError for another shape)."""
        if tuple(w.shape) != (self.d_out, self.d_in):
            raise ValueError(f"w: [{self.d_out}, {self.d_in}] is expected, not {list(w.shape)}")
        self.w.copy_(w)
        abi.mxfp8_requant_packed(_ptr(self.w), _ptr(self._q), _ptr(self._s), [(0, 0, 0, self.d_out, self.d_in)], _stream())
        self._weight_operands()

    def _weight_operands(self) -> None:
        """After a requantization: tiled scales of W, and W^T from the main weight."""
        abi.mxfp8_scale_relayout(_ptr(self._s), _ptr(self._s_tiled), [(0, 0, self.d_out, self.d_in // 32, 1)], _stream())
        abi.mxfp8_quantize(_ptr(self.w), abi.HM_F32, self.d_out, self.d_in, self.d_in, 0, 0, 32, 0, 0, 0, _ptr(self.wt.q),
                           self.wt.k, _ptr(self.wt.s), _stream())

    @_on_its_device
    def forward(self, x: torch.Tensor, res: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """x, res: bf16 [tokens][d_in], contiguous -> (y bf16 [tokens][d_out], h = x + res).
        Other shapes, types, layouts and devices are refused (ValueError), here and in backward."""
        for name, t in (("x", x), ("res", res)):
            if t is not None or name == "x":
                _need(name, t, (self.tokens, self.d_in), torch.bfloat16, self.gamma.device)
        st, d = _stream(), self.d_in
        abi.rmsnorm_mxfp8(_ptr(x), d, _ptr(res), _ptr(self.h), d, abi.HM_BF16, self.tokens, d, _ptr(self.gamma), self.eps,
                          self.block, _ptr(self.rstd), _ptr(self.x8.q), _ptr(self.x8.s), st)
        abi.mxfp8_gemm(_ptr(self.x8.q), d, _ptr(self.x8.s), _ptr(self._q), d, _ptr(self._s_tiled), self.tokens, self.d_out,
                       d, _ptr(self.y), self.d_out, abi.HM_BF16, False, st)
        return self.y, self.h

    @_on_its_device
    def backward(self, dy: torch.Tensor, dres: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """dy bf16 [tokens][d_out], dres bf16 [tokens][d_in] -> (dx, dgamma).  Adds dW to
        self.g and dgamma to self.dgamma, so several micro-batches make one step's gradient."""
        _need("dy", dy, (self.tokens, self.d_out), torch.bfloat16, self.gamma.device)
        if dres is not None:
            _need("dres", dres, (self.tokens, self.d_in), torch.bfloat16, self.gamma.device)
        st, m, k, n = _stream(), self.tokens, self.d_in, self.d_out
        abi.mxfp8_quantize(_ptr(dy), abi.HM_BF16, m, n, n, 0, 0, self.block, _ptr(self.dy8.q), self.dy8.k, _ptr(self.dy8.s),
                           _ptr(self.dyt8.q), self.dyt8.k, _ptr(self.dyt8.s), st)
        # norm(h)^T from h: the forward pass stored neither norm(h) nor its transpose
        abi.mxfp8_quantize(_ptr(self.h), abi.HM_BF16, m, k, k, _ptr(self.rstd), _ptr(self.gamma), self.block, 0, 0, 0,
                           _ptr(self.xt8.q), self.xt8.k, _ptr(self.xt8.s), st)
        abi.mxfp8_gemm(_ptr(self.dy8.q), self.dy8.k, _ptr(self.dy8.s), _ptr(self.wt.q), self.wt.k, _ptr(self.wt.s), m, k,
                       self.dy8.k, _ptr(self.dn), k, abi.HM_BF16, False, st)
        abi.mxfp8_gemm(_ptr(self.dyt8.q), self.dyt8.k, _ptr(self.dyt8.s), _ptr(self.xt8.q), self.xt8.k, _ptr(self.xt8.s), n,
                       k, self.dyt8.k, _ptr(self.g), k, abi.HM_F32, True, st)
        abi.rmsnorm_backward(_ptr(self.dn), k, _ptr(dres), _ptr(self.h), _ptr(self.dx), k, abi.HM_BF16, m, k,
                             _ptr(self.gamma), _ptr(self.rstd), _ptr(self.dgamma), self._summed, _ptr(self._ws),
                             self._ws.numel(), st)
        self._summed = True
        return self.dx, self.dgamma

    @_on_its_device
    def step(self, hp: "abi.hm_muon_hparams", max_norm: float = 1.0) -> torch.Tensor:
        """Clips dW and dgamma by their global norm, runs the Muon update of W (which requantizes
        it) and starts new gradients (zero_grad).  Returns (norm, coefficient) on the device; gamma
        is the caller's (AdamW on self.dgamma, say, before the next backward pass)."""
        stats = self.session.clip_grad_norm(max_norm, tensors=self._clip)
        self.session.run(hp, abi.HM_STAGE_ALL, torch.cuda.current_stream())
        self._weight_operands()
        self.zero_grad()
        return stats

    def close(self) -> None:
        self.session.close()
