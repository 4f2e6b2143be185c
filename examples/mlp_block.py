"""One gated MLP block of a transformer through the layer operators, in 16 bits and in MXFP8.

    h = x + residual
    y = rmsnorm(h) * g
    out = h + (silu(y @ w_gate.T) * (y @ w_up.T)) @ w_down.T

In 16 bits that is four calls: the norm with the residual's addition; the up product; the gate product with silu and
the multiplication in its epilogue; the down product with the addition of h in its epilogue.  In MXFP8 the norm and the
gate product write the 8-bit operands of the products that follow, and the weights are quantised once.

    python examples/mlp_block.py            # checks both against 64 bits, then times them
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import broadcast_implicit_gemm_gb300 as bg  # noqa: E402


def weights(hidden: int, inner: int, dtype=torch.bfloat16, seed: int = 0) -> dict:
    """Random weights of a block, of unit gain."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(rows, cols):
        return (torch.randn((rows, cols), generator=gen, device="cuda") / math.sqrt(cols)).to(dtype)

    return {"g": 1 + 0.1 * torch.randn((hidden,), generator=gen, device="cuda"),
            "gate": normal(inner, hidden), "up": normal(inner, hidden), "down": normal(hidden, inner)}


def quantised(w: dict) -> dict:
    """The same weights with the three matrices as MXFP8 (elements, scales); done once."""
    return {"g": w["g"], **{k: bg.mx_quantize(w[k]) for k in ("gate", "up", "down")}}


def block(x, residual, w: dict):
    """(out, h) in x's type (float16 or bfloat16)."""
    y, h = bg.rmsnorm(x, w["g"], residual=residual)
    up = bg.matmul(y, w["up"])
    z = bg.matmul(y, w["gate"], act=bg.ACT_SILU, other=up, combine=bg.COMBINE_MUL)
    return bg.matmul(z, w["down"], other=h), h


def block_mx(x, residual, w: dict):
    """(out, h) in x's type, the three products over MXFP8 operands; w from quantised()."""
    y, ys, h = bg.rmsnorm(x, w["g"], residual=residual, out_dtype=torch.float8_e4m3fn)
    up = bg.matmul_mx(y, ys, *w["up"], out_dtype=x.dtype)
    z, zs = bg.matmul_mx(y, ys, *w["gate"], act=bg.ACT_SILU, other=up, combine=bg.COMBINE_MUL,
                         out_dtype=torch.float8_e4m3fn)
    return bg.matmul_mx(z, zs, *w["down"], other=h, out_dtype=x.dtype), h


def block64(x, residual, w: dict, eps: float = 1e-6):
    """The block in 64 bits, of the 16-bit inputs and weights."""
    h = x.double() + residual.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w["g"].double()
    a = y @ w["gate"].double().t()
    z = a * torch.sigmoid(a) * (y @ w["up"].double().t())
    return h + z @ w["down"].double().t()


def _time(call, repeats: int = 20) -> float:
    """Microseconds per call, captured in a graph."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            call()
    graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(repeats):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / (4 * repeats)


def main() -> int:
    w = weights(512, 1408)
    x, r = torch.randn((2, 70, 512), device="cuda").to(torch.bfloat16)
    ref = block64(x, r, w)
    for name, got in (("bf16", block(x, r, w)[0]), ("mxfp8", block_mx(x, r, quantised(w))[0])):
        print(f"{name}: relative error against 64 bits {float((got.double() - ref).norm() / ref.norm()):.2e}")
    hidden, inner = 4096, 16384
    w = weights(hidden, inner)
    q = quantised(w)
    for tokens in (1, 64, 1024, 8192):
        x, r = torch.randn((2, tokens, hidden), device="cuda").to(torch.bfloat16)
        flops = 6 * tokens * hidden * inner
        a, b = _time(lambda: block(x, r, w)), _time(lambda: block_mx(x, r, q))
        print(f"{tokens} tokens, {hidden} x {inner}: bf16 {a:.1f} us ({flops / a / 1e6:.0f} TFLOP/s), "
              f"mxfp8 {b:.1f} us ({flops / b / 1e6:.0f} TFLOP/s)")
    return 0 if bg.bigemm_last_device_error() == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
