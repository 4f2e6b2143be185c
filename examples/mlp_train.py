"""The gated MLP block of mlp_block.py as training takes it: its forward pass keeps what the gradients need, and its
backward pass gives the gradients of everything that went in.

    h = x + residual
    y = norm(h)                                   # root-mean-square norm, or layer norm with a bias
    out = h + (silu(y @ w_gate.T) * (y @ w_up.T)) @ w_down.T

Forward: three calls (the norm with the residual's addition; both products of the gated layer with the activation and the
multiplication; the down product with h's addition).  Backward: three (the down product's gradients; the gated layer's;
the norm's, which adds the gradient that reaches h along the residual stream).

    python examples/mlp_train.py            # checks the gradients against 64 bits, then times a step
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import broadcast_implicit_gemm_gb300 as bg  # noqa: E402
import mlp_block  # noqa: E402


def weights(hidden: int, inner: int, dtype=torch.bfloat16, layer: bool = False, seed: int = 0) -> dict:
    """mlp_block's weights; with a layer norm's bias "b" too."""
    w = mlp_block.weights(hidden, inner, dtype, seed)
    if layer:
        w["b"] = 0.1 * torch.randn((hidden,), generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda")
    return w


def forward(x, residual, w: dict):
    """(out, what backward takes), in x's type (float16 or bfloat16)."""
    kept = {}
    if "b" in w:
        kept["mean"], kept["rstd"] = torch.empty((2, x.shape[0]), device=x.device)
        y, h = bg.layernorm(x, w["g"], w["b"], residual=residual, mean_out=kept["mean"], rstd_out=kept["rstd"])
    else:
        y, h = bg.rmsnorm(x, w["g"], residual=residual)
    gate, up = torch.empty((2, x.shape[0], w["gate"].shape[0]), dtype=x.dtype, device=x.device)
    z = bg.matmul_gated(y, w["gate"], w["up"], act=bg.ACT_SILU, gate_out=gate, up_out=up)
    kept.update(h=h, y=y, gate=gate, up=up, z=z)
    return bg.matmul(z, w["down"], other=h), kept


def backward(dout, kept: dict, w: dict) -> dict:
    """Gradients of x (and residual, which is the same), of the norm's weights and of the three matrices."""
    dz, ddown = bg.matmul_backward(dout, kept["z"], w["down"])
    dy, dgate, dup = bg.matmul_gated_backward(dz, kept["y"], w["gate"], w["up"], kept["gate"], kept["up"], act=bg.ACT_SILU)
    grads = {"gate": dgate, "up": dup, "down": ddown}
    if "b" in w:
        grads["x"], grads["g"], grads["b"] = bg.layernorm_backward(dy, kept["h"], kept["mean"], kept["rstd"], w["g"], dsum=dout)
    else:
        grads["x"], grads["g"] = bg.rmsnorm_backward(dy, kept["h"], w["g"], dsum=dout)
    return grads


def gradients64(dout, x, residual, w: dict, eps: float | None = None) -> dict:
    """The same in 64 bits, by torch's differentiation of the block."""
    leaf = {k: v.double().requires_grad_() for k, v in w.items()}
    a = x.double().requires_grad_()
    h = a + residual.double()
    if "b" in w:
        y = torch.nn.functional.layer_norm(h, h.shape[-1:], leaf["g"], leaf["b"], 1e-5 if eps is None else eps)
    else:
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + (1e-6 if eps is None else eps)) * leaf["g"]
    g = y @ leaf["gate"].t()
    out = h + (g * torch.sigmoid(g) * (y @ leaf["up"].t())) @ leaf["down"].t()
    names = ["x", *leaf]
    return dict(zip(names, torch.autograd.grad(out, [a, *leaf.values()], dout.double())))


def main() -> int:
    for layer in (False, True):
        w = weights(512, 1408, layer=layer)
        x, r, d = torch.randn((3, 70, 512), device="cuda").to(torch.bfloat16)
        out, kept = forward(x, r, w)
        got, ref = backward(d, kept, w), gradients64(d, x, r, w)
        print("layer norm:" if layer else "rms norm:",
              ", ".join(f"d{k} {float((got[k].double() - ref[k]).norm() / ref[k].norm()):.1e}" for k in ref))
    hidden, inner = 4096, 16384
    w = weights(hidden, inner)
    for tokens in (64, 1024, 8192):
        x, r, d = torch.randn((3, tokens, hidden), device="cuda").to(torch.bfloat16)

        def step():
            _, kept = forward(x, r, w)
            return backward(d, kept, w)
        us = mlp_block._time(step, 5)
        print(f"{tokens} tokens, {hidden} x {inner}: forward and backward {us:.0f} us "
              f"({18 * tokens * hidden * inner / us / 1e6:.0f} TFLOP/s)")
    return 0 if bg.bigemm_last_device_error() == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
