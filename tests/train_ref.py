"""64-bit forms of the layer norm, the norms' gradients, the gated products and the products' gradients, on the device of
their inputs, and their error bounds.

U = 2^-24 is half a step of fp32 at 1.  A sum in fp32 whose terms pass through at most n additions is off by at most
n U of the sum of magnitudes.

Sums over a row: a thread adds at most 16 elements (8 of every 4096 for rows beyond the registers), five shuffles join a
warp, five more or 16 additions the warps: n = cols / 512 + 40.  Sums over all rows: a thread adds the rows of its block
(at least 152 blocks where there are as many rows; runs of long rows are no longer), a few warps of a block join, and
then at most 1216 rows of partial sums by eight warps: n = rows / 100 + 180.

Each other operation (product, difference, conversion) is off by U of its result; a root's reciprocal by 4 U (2 ulp)."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def row_adds(cols):
    return cols / 512 + 40


def column_adds(rows):
    return rows / 100 + 180


def check(got, ref, d, what=""):
    """got is ref within d, and a rounding to its type."""
    assert got.shape == ref.shape, what
    assert bool(torch.isfinite(got).all()), what
    bound = d + HALF[got.dtype] * (ref.abs() + d) + TINY[got.dtype]
    over = ((got.double() - ref).abs() / bound).nan_to_num()
    assert float(over.max() if over.numel() else 0) <= 1, f"{what}: {float(over.max()):.3f} of the bound at {int(over.argmax())}"


def layernorm64(x, r, w, b, eps):
    """(y, its bound, h, mean, its bound, rstd, its bound)."""
    h = x.double() if r is None else x.double() + r.double()
    cols, n = h.shape[1], row_adds(h.shape[1])
    m = h.mean(-1, keepdim=True)
    d = h - m
    v = (d * d).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(v + eps)
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if w is None else w.double()
    y = d * rstd * w + (0 if b is None else b.double())
    em = (n + 4) * U * h.abs().mean(-1, keepdim=True)           # of the mean
    ed = U * h.abs() + em + U * d.abs()                         # of h - mean
    ev = (2 * d.abs() * ed + ed * ed).mean(-1, keepdim=True) + (n + 8) * U * v
    er = rstd * (0.5 * ev / (v + eps) + (ev / (v + eps)) ** 2 + 6 * U)
    ey = w.abs() * (ed * (rstd + er) + d.abs() * er) + 4 * U * (d * rstd * w).abs() + 2 * U * y.abs()
    return y, ey, h, m[:, 0], em[:, 0], rstd[:, 0], er[:, 0]


def layernorm_backward64(dout, x, mean, rstd, w, dsum):
    """{name: (value, bound)} of dx, dw and db; mean and rstd are inputs."""
    d, x = dout.double(), x.double()
    rows, cols = x.shape
    n, q = row_adds(cols), column_adds(rows)
    m, r = mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if w is None else w.double()
    xh, g = (x - m) * r, d * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    e1, e2 = (n + 3) * U * g.abs().mean(-1, keepdim=True), (n + 6) * U * (g * xh).abs().mean(-1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    size = g.abs() + c1.abs() + (xh * c2).abs()
    e = r * (e1 + xh.abs() * e2 + 7 * U * size)
    if dsum is not None:
        dx = dx + dsum.double()
        e = e + U * dx.abs()
    return {"dx": (dx, e), "dw": ((d * xh).sum(0), (q + 4) * U * (d * xh).abs().sum(0)),
            "db": (d.sum(0), q * U * d.abs().sum(0))}


def rmsnorm_backward64(dout, x, w, eps, dsum):
    d, x = dout.double(), x.double()
    rows, cols = x.shape
    n, q = row_adds(cols), column_adds(rows)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if w is None else w.double()
    xh, g = x * r, d * w
    c2 = (g * xh).mean(-1, keepdim=True)
    er = (n / 2 + 6) * U                                        # of r, relative
    e2 = 3 * er * c2.abs() + (n + 6) * U * (g * xh).abs().mean(-1, keepdim=True)
    dx = r * (g - xh * c2)
    size = g.abs() + (xh * c2).abs()
    e = r * (xh.abs() * e2 + (er + 7 * U) * size)
    if dsum is not None:
        dx = dx + dsum.double()
        e = e + U * dx.abs()
    return {"dx": (dx, e), "dw": ((d * xh).sum(0), ((q + 4) * U + er) * (d * xh).abs().sum(0))}


def act64(kind, z):
    """(act(z), its slope)."""
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p * (1 + z * (1 - p) * c * (1 + 3 * 0.044715 * z * z))
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    return z, torch.ones_like(z)


# Products.  As layer_ref derives: an instruction's 16 products and the accumulator are cut short by 2^-23 of a partial
# sum, at most S, twice; so a sum of L products is off by (L / 16 + 9) 2^-22 S, S the sum of magnitudes.
# Activations: an error of 2^-19 of max(|z|, 1), slopes at most 1.13; slopes are off by 2^-18 (a quotient of 2 ulp and an
# exponential whose argument is off by |z| ulp, times factors of at most 10 where they are not negligible).

def product_error(L, S):
    return (L / 16 + 9) * 2.0 ** -22 * S


def gated64(x, wg, wu, bg, bu, act):
    """{name: (value, bound)} of y, g and u."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    both = []
    for w, b in ((wg, bg), (wu, bu)):
        z, e = x @ w.T, product_error(K, x.abs() @ w.abs().T)
        if b is not None:
            z = z + b.double()
            e = e + 2 * U * (z.abs() + b.double().abs())
        both.append((z, e))
    (g, eg), (u, eu) = both
    a = act64(act, g)[0]
    ea = 1.13 * eg + 2.0 ** -19 * g.abs().clamp(min=1) * (act not in ("relu", "none"))
    y = a * u
    return {"y": (y, ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * y.abs()), "g": (g, eg), "u": (u, eu)}


def product_backward64(dout, x, w):
    """{name: (value, bound)} of dx, dw and db of one product of d (its own error: ed)."""
    d, x, w = dout.double(), x.double(), w.double()
    M, N = d.shape
    return {"dx": (d @ w, product_error(N + 512, d.abs() @ w.abs())), "dw": (d.T @ x, product_error(M, d.abs().T @ x.abs())),
            "db": (d.sum(0), column_adds(M) * U * d.abs().sum(0))}


def gated_backward64(dout, x, wg, wu, g, u, act):
    """{name: (value, bound)}: dg and du are off by the slopes' error and a rounding to the operands' type each."""
    kind = x.dtype
    d, x, wg, wu, g, u = (t.double() for t in (dout, x, wg, wu, g, u))
    M, N = d.shape
    a, s = act64(act, g)
    smooth = act not in ("relu", "none")
    dg, du = d * u * s, d * a
    eg = (d * u).abs() * 2.0 ** -18 * smooth + 3 * U * dg.abs()
    eu = d.abs() * 2.0 ** -19 * g.abs().clamp(min=1) * smooth + 2 * U * du.abs()
    n = column_adds(M)
    out = {"dbg": (dg.sum(0), eg.sum(0) + n * U * dg.abs().sum(0)), "dbu": (du.sum(0), eu.sum(0) + n * U * du.abs().sum(0))}
    eg = eg + HALF[kind] * dg.abs() + TINY[kind]
    eu = eu + HALF[kind] * du.abs() + TINY[kind]
    S = dg.abs() @ wg.abs() + du.abs() @ wu.abs()
    out["dx"] = (dg @ wg + du @ wu, eg @ wg.abs() + eu @ wu.abs() + product_error(2 * N + 640, S))
    out["dwg"] = (dg.T @ x, eg.T @ x.abs() + product_error(M, dg.abs().T @ x.abs()))
    out["dwu"] = (du.T @ x, eu.T @ x.abs() + product_error(M, du.abs().T @ x.abs()))
    return out


def check_norm(got, ref, roundings, what=""):
    """The 2-norm of the error of independent roundings to got's type, each of at most half a step and of a third of its
    square on average, with a half on top: an error in a few elements that each element's bound would hide."""
    if ref.numel() < 2000:
        return
    rel = float((got.double() - ref).norm() / ref.norm().clamp(min=1e-300))
    most = 1.5 * HALF[got.dtype] * math.sqrt(roundings / 3)
    assert rel <= most, f"{what}: 2-norm {rel:.3e}, at most {most:.3e}"
