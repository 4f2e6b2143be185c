"""The layer operators' 64-bit forms on the GPU, for sizes at which layer_ref's take too long, and their bounds.

matmul: as layer_ref derives them, with the pieces that the kernels sum: 512 products of 16-bit operands, 2048 of MXFP8
ones.  The 2-norm of a 32-bit output's error is bounded besides (test_gpu_matmul_sums derives it), so that an error which
each element's bound would hide is seen."""
import math

import torch

from tests.layer_ref import TINY, U

MX = torch.float8_e4m3fn
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "mx": MX}


def rand(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale


def strided(t, pad, dtype):
    """The matrix as columns of a wider tensor, NaN in the others."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device="cuda").to(dtype)
    big[:, : t.shape[1]] = t.to(dtype)
    return big[:, : t.shape[1]]


def codes_of(scale, rows, cols):
    """[rows, groups] of the rows' whole blocks, the padding's too."""
    a, b = -(-rows // 128), -(-cols // 128)
    return scale.view(torch.uint8).reshape(a, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(a * 128, b * 4)[:rows].int()


def decoded(q, scale):
    rows, cols = q.shape
    s = torch.pow(2.0, codes_of(scale, rows, cols).double() - 127)
    return q.double() * s.repeat_interleave(32, 1)[:, :cols]


def act64(kind, z):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def product64(x, w, bias, act, other, combine, pieces, mx):
    """(reference, bound before the output's rounding) of the product of 64-bit matrices; pieces: K summed in them."""
    K = x.shape[1]
    z, S = x @ w.T, x.abs() @ w.abs().T
    step, piece = (32, 2048) if mx else (16, 512)
    if pieces:
        d = ((min(K, piece) / step + 1) * 2.0 ** -22 + (K / piece + 8) * 2.0 ** -24) * S
    else:
        d = (K / step + 9) * 2.0 ** -22 * S
    del S
    if bias is not None:
        z = z + bias.double()
        d = d + 2.0 ** -23 * (z.abs() + bias.double().abs())
    y = act64(act, z)
    if act != "none":
        d = 1.13 * d + 2.0 ** -19 * z.abs().clamp(min=1) * (act != "relu")
    if combine == "add":
        y = y + other.double()
        d = d + 2.0 ** -23 * y.abs()
    elif combine == "mul":
        y = y * other.double()
        d = d * other.double().abs() + 2.0 ** -23 * y.abs()
    return y, d


def check_float(got, ref, d, what=""):
    bound = d + U[got.dtype] * (ref.abs() + d) + TINY[got.dtype]
    over = (got.double() - ref).abs() / bound
    assert bool((over <= 1).all()), f"{what}: worst {float(over.max()):.3f} of the bound at {divmod(int(over.argmax()), ref.shape[1])}"


def code_of(amax):
    """E8M0 code of the smallest power of two s >= 2^-127 with amax <= 448 s, of 64-bit values."""
    m, e = torch.frexp(amax / 448)
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    return torch.where(amax > 0, e, torch.full_like(e, -127)) + 127


def group_max(v):
    rows, cols = v.shape
    full = torch.zeros((rows, -(-cols // 128) * 128), dtype=v.dtype, device=v.device)
    full[:, :cols] = v.abs()
    return full.view(rows, -1, 32).amax(-1)


def check_mx(q, scale, ref, d, what=""):
    rows, cols = ref.shape
    code = codes_of(scale, rows, cols)
    groups = -(-cols // 32)
    assert not bool(code[:, groups:].any()), f"{what}: codes past the last column"
    top, off = group_max(ref), group_max(d)
    assert bool(((code >= code_of((top - off).clamp(min=0))) & (code <= code_of(top + off)))[:, :groups].all()), f"{what}: scales"
    s = torch.pow(2.0, code.double() - 127).repeat_interleave(32, 1)[:, :cols]
    e = torch.floor(torch.log2(((ref.abs() + d) / s).clamp(min=2.0 ** -6))).clamp(-6, 8)
    bound = d + 0.5 * s * torch.pow(2.0, e - 3) * (1 + 1e-9)
    over = (q.double() * s - ref).abs() / bound
    assert bool((over <= 1).all()), f"{what}: worst {float(over.max()):.3f} of the bound at {divmod(int(over.argmax()), cols)}"
