"""A few training steps of an RMS norm and a linear layer on MXFP8 operands:
norm -> product -> loss -> gradient products -> clipping -> Muon update ->
requantization, all in the library's kernels.

    python examples/norm_linear_step.py [--tokens 512] [--d-in 1024] [--d-out 768] [--steps 10]

The target is a fixed linear map of the normed input, so the loss falls.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from head_muon_mxfp8_gb300 import abi  # noqa: E402
from head_muon_mxfp8_gb300.linear import NormLinear  # noqa: E402


def train(tokens: int = 512, d_in: int = 1024, d_out: int = 768, steps: int = 10, lr: float = 0.2, seed: int = 0):
    """Returns the losses (one per step) and the (norm, coefficient) pairs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(tokens, d_in, generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn(tokens, d_in, generator=g, device="cuda").to(torch.bfloat16)
    h = (x.float() + res.float())
    normed = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-5)
    target = normed @ (torch.randn(d_out, d_in, generator=g, device="cuda") / d_in ** 0.5).t()
    layer = NormLinear(tokens, d_in, d_out)
    layer.load_weight(torch.randn(d_out, d_in, generator=g, device="cuda") / d_in ** 0.5)
    gm, gv = torch.zeros(d_in, device="cuda"), torch.zeros(d_in, device="cuda")
    losses, stats = [], []
    for step in range(steps):
        y, _ = layer.forward(x, res)
        err = y.float() - target
        losses.append(err.square().mean())
        layer.backward((err * (2.0 / err.numel())).to(torch.bfloat16))
        hp = abi.hm_muon_hparams(lr * (1 - step / steps), 0.9, 0.0, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, 0)
        stats.append(layer.step(hp, max_norm=1.0).clone())
        abi.adamw_update_flat(layer.gamma.data_ptr(), layer.dgamma.data_ptr(), abi.HM_F32, gm.data_ptr(), gv.data_ptr(),
                              d_in, abi.hm_adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.0, step + 1),
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    if abi.hm_device_error():
        raise RuntimeError("a device-side wait gave up")
    layer.close()
    return [float(v) for v in losses], [v.tolist() for v in stats]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--d-in", type=int, default=1024)
    ap.add_argument("--d-out", type=int, default=768)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    losses, stats = train(a.tokens, a.d_in, a.d_out, a.steps)
    for i, (loss, (norm, coef)) in enumerate(zip(losses, stats)):
        print(f"step {i}: loss {loss:.4f}  gradient norm {norm:.3e}  coefficient {coef:.3f}")


if __name__ == "__main__":
    main()
