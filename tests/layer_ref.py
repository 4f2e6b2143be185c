"""Plain 64-bit forms of the transformer-layer operators, and their error bounds.

matmul: the tensor core adds the products of one instruction (16 elements of K
in 16 bits, 32 in 8) to an fp32 accumulator, each addition cut short by at most
2^-23 of a partial sum, itself at most S = sum |x w|; twice that is allowed for
the sum within the instruction:  d = (steps * 2^-22) S, steps = K / 16 or
K / 32.  A 32-bit output sums at most 1024 elements that way and adds the
pieces, and the CTAs' shares (at most 8), in fp32: (K / 1024 + 8) 2^-24 S more.
The activations' slopes are at most 1.13 and their own error at most 2^-19 of
max(|z|, 1) (a quotient of 2 ulp over an exponential whose argument is off by
2 ulp of at most 30, where it matters).  Then the output's rounding.

MXFP8 outputs: the code may be that of any magnitude within the group's error of
the reference's; given the code, an element is off by its error and half a step.
"""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def scale_index(rows, cols):
    r = np.arange(rows)[:, None]
    g = np.arange(-(-cols // 32))[None, :]
    return r // 128, g // 4, r % 32, (r % 128) // 32, g % 4


def decode(q, scale):
    """Values of an MXFP8 matrix in 64 bits."""
    rows, cols = q.shape
    code = scale.view(torch.uint8).cpu().numpy().reshape(-(-rows // 128), -(-cols // 128), 32, 4, 4)
    code = code[scale_index(rows, cols)].astype(np.int64)
    f = np.where(code == 255, np.nan, np.ldexp(1.0, np.minimum(code, 254) - 127))
    return q.cpu().float().double().numpy() * np.repeat(f, 32, axis=1)[:, :cols]


def codes_of(scale, rows, cols):
    code = scale.view(torch.uint8).cpu().numpy().reshape(-(-rows // 128), -(-cols // 128), 32, 4, 4)
    return code[scale_index(rows, cols)].astype(np.int64)


def code_of(amax):
    """E8M0 code of the smallest power of two s >= 2^-127 with amax <= 448 s."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0))
    for _ in range(2):   # log2's own rounding
        e = np.where(amax > 448.0 * 2.0 ** e, e + 1, e)
        e = np.where((amax <= 448.0 * 2.0 ** (e - 1)), e - 1, e)
    return np.clip(e, -127, 127).astype(np.int64) + 127


def group_max(v):
    rows, cols = v.shape
    full = np.zeros((rows, -(-cols // 32) * 32))
    full[:, :cols] = np.abs(v)
    return full.reshape(rows, -1, 32).max(-1)


def act64(kind, z):
    if kind == "relu":
        return np.maximum(z, 0)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(torch.from_numpy(z / math.sqrt(2))).numpy())
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        with np.errstate(over="ignore"):
            return z / (1 + np.exp(-z))
    return z


def product64(x, w, bias, act, other, combine, out_dtype, mx):
    """(reference, bound before the output's rounding) of the product; x and w 64-bit arrays."""
    K = x.shape[1]
    z, S = x @ w.T, np.abs(x) @ np.abs(w).T
    step = 32 if mx else 16
    if out_dtype == torch.float32:
        d = (min(K, 1024) / step + 1) * 2.0 ** -22 * S + (K / 1024 + 8) * 2.0 ** -24 * S
    else:
        d = (K / step + 9) * 2.0 ** -22 * S
    if bias is not None:
        z = z + bias
        d = d + 2.0 ** -23 * (np.abs(z) + np.abs(bias))
    y = act64(act, z)
    if act != "none":
        d = 1.13 * d + 2.0 ** -19 * np.maximum(np.abs(z), 1) * (act != "relu")
    if combine == "add":
        y = y + other
        d = d + 2.0 ** -23 * np.abs(y)
    elif combine == "mul":
        y = y * other
        d = d * np.abs(other) + 2.0 ** -23 * np.abs(y)
    return y, d


def check_float(got, ref, d, what=""):
    u, tiny = U[got.dtype], TINY[got.dtype]
    g = got.cpu().double().numpy()
    bound = d + u * (np.abs(ref) + d) + tiny
    err = np.abs(g - ref)
    assert np.isfinite(g).all(), what
    assert (err <= bound).all(), f"{what}: worst {np.max(err / bound):.3f} of the bound"


def check_mx(q, scale, ref, d, what=""):
    rows, cols = ref.shape
    code = codes_of(scale, rows, cols)
    top, off = group_max(ref), group_max(d * np.ones_like(ref))
    lo, hi = code_of(np.maximum(top - off, 0)), code_of(top + off)
    assert ((code >= lo) & (code <= hi)).all(), f"{what}: scales"
    v = decode(q, scale)
    s = np.repeat(np.ldexp(1.0, code - 127), 32, axis=1)[:, :cols]
    m = np.abs(ref) + d
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(m / s, 2.0 ** -6)))
    half = 0.5 * s * 2.0 ** (np.clip(e, -6, 8) - 3)
    err = np.abs(v - ref)
    assert (err <= d + half * (1 + 1e-9)).all(), f"{what}: worst {np.max(err / (d + half)):.3f} of the bound"


def padding_codes_are_zero(scale, rows, cols):
    """The codes past the last column of the rows' last block, and those of rows past the last, are as allocated."""
    a, b = -(-rows // 128), -(-cols // 128)
    code = scale.view(torch.uint8).cpu().numpy().reshape(a, b, 32, 4, 4)
    full = code.transpose(0, 3, 2, 1, 4).reshape(a * 128, b * 4)
    return not full[rows:].any() and not full[:, -(-cols // 32):].any()
