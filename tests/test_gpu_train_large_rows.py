"""More than 2^31 elements in the layer norm, the gated layer and the gradients, every output NaN before the call, so that
a row that no thread writes shows: all rows are zero but some at both ends and where the offsets pass 2^30 and 2^31
elements, and the whole result is known from those."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)


def unwritten(*shape, dtype=BF):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def chosen(rows, cols):
    """Rows that are not zero."""
    at = {*range(3), *range(rows - 3, rows)}
    for border in (2 ** 30 // cols, 2 ** 31 // cols):
        at |= {border - 1, border, border + 1}
    return torch.tensor(sorted(at), device="cuda")


def matrix(rows, cols, at, seed):
    t = torch.zeros((rows, cols), dtype=BF, device="cuda")
    t[at] = rand((len(at), cols), seed)
    return t


def zero_elsewhere(t, at, what):
    """Every other row is zero (NaN is not)."""
    edges = [-1, *at.tolist(), t.shape[0]]
    for a, b in zip(edges, edges[1:]):
        for i in range(a + 1, b, 1 << 17):
            assert not t[i: min(b, i + (1 << 17))].any(), f"{what}: rows {i} to {b}"


def quiet():
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0


@pytest.mark.parametrize("rows,cols", [(270_001, 8000), (1_200_003, 1801), (133_001, 16392)])
def test_norms(rows, cols):
    """On the 16-byte grid, off it, and rows that a cluster shares."""
    assert rows * cols > 2 ** 31
    at = chosen(rows, cols)
    x, d = matrix(rows, cols, at, 1), matrix(rows, cols, at, 2)
    mean, rstd, out = unwritten(rows, dtype=torch.float32), unwritten(rows, dtype=torch.float32), unwritten(rows, cols)
    bg.layernorm(x, out=out, mean_out=mean, rstd_out=rstd)
    quiet()
    ref, ey, _, m, em, r, er = tr.layernorm64(x[at], None, None, None, 1e-5)
    tr.check(out[at], ref, ey, "y")
    tr.check(mean[at], m, em, "mean")
    tr.check(rstd[at], r, er, "rstd")
    zero_elsewhere(out, at, "y")
    zero_elsewhere(mean[:, None], at, "mean")
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[at] = False
    assert float((rstd[others].double() - 1e-5 ** -0.5).abs().max()) < 8 * tr.U * 1e-5 ** -0.5
    for layer in (True, False):
        dw, db = unwritten(cols, dtype=torch.float32), unwritten(cols, dtype=torch.float32)
        out.fill_(float("nan"))
        if layer:
            bg.layernorm_backward(d, x, mean, rstd, dx=out, dweight=dw, dbias=db)
            ref = tr.layernorm_backward64(d[at], x[at], mean[at], rstd[at], None, None)
        else:
            bg.rmsnorm_backward(d, x, dx=out, dweight=dw)
            ref = tr.rmsnorm_backward64(d[at], x[at], None, 1e-6, None)
        quiet()
        tr.check(out[at], *ref["dx"], "dx")
        zero_elsewhere(out, at, "dx")
        tr.check(dw, *ref["dw"], "dw")           # (the other rows add zeros)
        if layer:
            tr.check(db, *ref["db"], "db")


def test_gated_layer():
    """140 000 tokens by 16 384 channels, 2.3e9 elements."""
    M, N, K = 140_001, 16384, 64
    at = chosen(M, N)
    x, wg, wu = matrix(M, K, at, 1), rand((N, K), 2) * 0.125, rand((N, K), 3) * 0.125
    kept = {name: unwritten(M, N) for name in ("y", "g", "u")}
    bg.matmul_gated(x, wg, wu, out=kept["y"], gate_out=kept["g"], up_out=kept["u"])
    quiet()
    ref = tr.gated64(x[at], wg, wu, None, None, "silu")
    for name, t in kept.items():
        tr.check(t[at], *ref[name], name)
        zero_elsewhere(t, at, name)
    g, u, d = kept["g"], kept["u"], kept.pop("y").zero_()
    d[at] = rand((len(at), N), 4)
    dx, dwg, dwu = unwritten(M, K), unwritten(N, K), unwritten(N, K)
    dbg, dbu = unwritten(N, dtype=torch.float32), unwritten(N, dtype=torch.float32)
    bg.matmul_gated_backward(d, x, wg, wu, g, u, dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=dbg, dbias_up=dbu)
    quiet()
    ref = tr.gated_backward64(d[at], x[at], wg, wu, g[at], u[at], "silu")
    tr.check(dx[at], *ref["dx"], "dx")
    zero_elsewhere(dx, at, "dx")
    for name, t in (("dwg", dwg), ("dwu", dwu), ("dbg", dbg), ("dbu", dbu)):
        tr.check(t, *ref[name], name)
    for t in (dx, dwg, dbg):
        t.fill_(float("nan"))
    bg.matmul_backward(d, x, wg, dx=dx, dw=dwg, dbias=dbg)
    quiet()
    ref = tr.product_backward64(d[at], x[at], wg)
    tr.check(dx[at], *ref["dx"], "dx")
    zero_elsewhere(dx, at, "dx")
    tr.check(dwg, *ref["dw"], "dw")
    tr.check(dbg, *ref["db"], "db")
