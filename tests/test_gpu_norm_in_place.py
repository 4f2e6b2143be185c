"""Outputs of the norms that take the place of their inputs, rows on the 16-byte grid and off it, of a warp, a block, a
cluster, and longer ones: the same bits as in a matrix of the same layout elsewhere (off the grid the layout of the rows
decides which elements a thread adds up)."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

SIZES = [(2000, 264), (700, 333), (400, 4096), (200, 9999), (30, 16392), (60, 20001), (9, 70008), (9, 70001)]


def rand(shape, seed, pad):
    rows, cols = shape
    t = torch.randn((rows, cols + pad), generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()
    return t[:, pad // 2: pad // 2 + cols]


def copied(t):
    """The same matrix, with the same rows, elsewhere."""
    big = t._base.clone() if t._base is not None else t.clone()
    return big.as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("pad", [0, 16, 3])
@pytest.mark.parametrize("same", ["x", "residual"])
def test_layernorm(rows, cols, pad, same):
    x, r = rand((rows, cols), 1, pad), rand((rows, cols), 2, pad)
    for both in (False, True):
        y, h = bg.layernorm(x, residual=r, out=copied(x), sum_out=copied(x) if both else None)
        a, b = copied(x), copied(r)
        out = a if same == "x" else b
        other = (b if same == "x" else a) if both else None
        y2, h2 = bg.layernorm(a, residual=b, out=out, sum_out=other)
        assert y2 is out and torch.equal(y, y2) and torch.equal(h, h2)
    a = copied(x)
    assert torch.equal(bg.layernorm(a, out=a), bg.layernorm(x, out=copied(x)))


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("pad", [0, 16, 3])
@pytest.mark.parametrize("same", ["dout", "x", "dsum"])
def test_gradients(rows, cols, pad, same):
    t = {"x": rand((rows, cols), 1, pad), "dout": rand((rows, cols), 2, pad), "dsum": rand((rows, cols), 3, pad)}
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    bg.layernorm(t["x"], mean_out=mean, rstd_out=rstd)

    layer, rms = (lambda t, dx: bg.layernorm_backward(t["dout"], t["x"], mean, rstd, dsum=t["dsum"], dx=dx),
                  lambda t, dx: bg.rmsnorm_backward(t["dout"], t["x"], dsum=t["dsum"], dx=dx))
    for call in (layer, rms):
        want = call(t, copied(t["x"]))
        mine = {k: copied(v) for k, v in t.items()}
        got = call(mine, mine[same])
        assert got[0] is mine[same] and all(torch.equal(a, b) for a, b in zip(want, got))
