"""GPU parity of the layer norm and of the norms' gradients against their 64-bit definitions (train_ref has the bounds)."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref as lr
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "mx": torch.float8_e4m3fn}


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def strided(t, pad, dtype, offset=0):
    """The matrix as columns of a wider tensor, NaN in the others."""
    big = torch.full((t.shape[0], t.shape[1] + pad + offset), float("nan"), device="cuda").to(dtype)
    big[:, offset: offset + t.shape[1]] = t.to(dtype)
    return big[:, offset: offset + t.shape[1]]


def untouched(t, offset):
    return bool(torch.isnan(t._base[:, offset + t.shape[1]:]).all()) and bool(torch.isnan(t._base[:, :offset]).all())


def norm_case(rows, cols, kind="bf16", out="same", residual=True, affine=True, pad=0, offset=0, eps=1e-5, seed=1, size=1.0,
              level=0.3, stats=True):
    x = strided((rand((rows, cols), seed) + level) * size, pad, TD[kind], offset)
    r = strided(rand((rows, cols), seed + 1) * size, pad, TD[kind], offset) if residual else None
    w, b = (1 + 0.2 * rand((cols,), seed + 2), rand((cols,), seed + 3)) if affine else (None, None)
    odt = TD[kind] if out == "same" else TD[out]
    h = strided(torch.zeros((rows, cols), device="cuda"), pad, TD[kind], offset) if residual else None
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2)) if stats else (None, None)
    y = None if out == "mx" else strided(torch.zeros((rows, cols), device="cuda"), pad, odt, offset)
    got = bg.layernorm(x, w, b, residual=r, eps=eps, out_dtype=odt, out=y, sum_out=h, mean_out=mean, rstd_out=rstd)
    torch.cuda.synchronize()
    ref, ey, hs, m, em, rs, er = tr.layernorm64(x, r, w, b, eps)
    what = f"{rows}x{cols} {kind}->{out}"
    if residual:
        assert got[-1] is h
        tr.check(h, hs, tr.U * hs.abs(), what + " sum")
        assert untouched(h, offset)
    if stats:
        tr.check(mean, m, em, what + " mean")
        tr.check(rstd, rs, er, what + " rstd")
    if out == "mx":
        lr.check_mx(got[0], got[1], ref.cpu().numpy(), ey.cpu().numpy(), what)
        assert lr.padding_codes_are_zero(got[1], rows, cols)
    else:
        tr.check(y, ref, ey, what)
        assert untouched(y, offset)


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 31, 32, 33, 127, 128, 255, 256, 257, 511, 513, 1000, 1023, 1025, 2049, 4096, 4104, 8192,
                                  16384, 16392, 20001])
@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("f16", "mx"), ("bf16", "f32"), ("f32", "same")])
def test_widths(cols, kind, out):
    norm_case(5, cols, kind, out, seed=cols)


@pytest.mark.parametrize("rows", [1, 2, 31, 129, 700])
@pytest.mark.parametrize("cols", [200, 520])
@pytest.mark.parametrize("out", ["same", "mx"])
def test_rows(rows, cols, out):
    norm_case(rows, cols, "bf16", out, seed=rows)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "f32", "mx"])
@pytest.mark.parametrize("residual,affine,stats", [(False, False, True), (True, False, False), (False, True, False), (True, True, True)])
def test_forms(kind, out, residual, affine, stats):
    norm_case(9, 776, kind, out, residual, affine, stats=stats)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("out", ["same", "mx", "f32"])
@pytest.mark.parametrize("cols", [200, 648, 17003])
def test_strides(pad, offset, out, cols):
    norm_case(40, cols, "f16", out, pad=pad, offset=offset)


def test_many_rows_per_block():
    """More rows than one wave of blocks holds, on and off the grid."""
    norm_case(5000, 1000, "bf16", seed=3)
    norm_case(5001, 203, "f16", seed=4)
    norm_case(1300, 4099, "bf16", seed=5, residual=False)


def test_rows_far_from_zero():
    """The variance keeps its digits where the mean is large (a difference of squares' means would lose them all)."""
    norm_case(6, 4096, "f32", level=300.0, residual=False, affine=False, seed=1)
    norm_case(6, 20000, "f32", level=300.0, residual=False, affine=False, seed=2)
    norm_case(6, 130, "f32", level=-300.0, residual=False, affine=False, seed=3)


def test_constant_rows():
    x = torch.full((3, 1000), 0.25, dtype=torch.float16, device="cuda")
    b = rand((1000,), 1)
    y = bg.layernorm(x, None, b, out_dtype=torch.float32)
    assert torch.equal(y, b.expand_as(y))                # the mean of a constant is exact in fp32 here
    assert bg.layernorm(x[:0]).shape == (0, 1000)


def test_nan_stays_in_its_row():
    x = rand((6, 300), 1).bfloat16()
    clean = bg.layernorm(x)
    x[2, 17] = float("nan")
    x[4, 299] = float("inf")
    got = bg.layernorm(x)
    keep = [0, 1, 3, 5]
    assert torch.isnan(got[2]).all() and torch.isnan(got[4]).all() and torch.equal(got[keep], clean[keep])


def test_sum_in_place():
    for cols in (768, 20000):
        x, r = rand((20, cols), 1).half(), rand((20, cols), 2).half()
        y, h = bg.layernorm(x, residual=r)
        y2, h2 = bg.layernorm(x, residual=r, sum_out=r)
        assert h2 is r and torch.equal(h, r) and torch.equal(y, y2)


# --------------------------------------------------------------------- gradients

def back_case(which, rows, cols, kind="bf16", dsum=True, affine=True, pad=0, offset=0, seed=1, inplace=None, size=1.0):
    x = strided((rand((rows, cols), seed) + 0.3) * size, pad, TD[kind], offset)
    d = strided(rand((rows, cols), seed + 1) * 0.1, pad, TD[kind], offset)
    s = strided(rand((rows, cols), seed + 2) * 0.1, pad, TD[kind], offset) if dsum else None
    w = 1 + 0.2 * rand((cols,), seed + 3) if affine else None
    out = {"dout": d, "dsum": s}.get(inplace)
    if out is None:
        out = strided(torch.zeros((rows, cols), device="cuda"), pad, TD[kind], offset)
    if which == "layer":
        _, _, _, m, _, r, _ = tr.layernorm64(x, None, None, None, 1e-5)
        m, r = m.float(), r.float()
        ref = tr.layernorm_backward64(d, x, m, r, w, s)
        got = bg.layernorm_backward(d, x, m, r, w, dsum=s, dx=out)
    else:
        ref = tr.rmsnorm_backward64(d, x, w, 1e-6, s)
        got = bg.rmsnorm_backward(d, x, w, eps=1e-6, dsum=s, dx=out)
    torch.cuda.synchronize()
    assert got[0] is out and untouched(out, offset)
    for name, g in zip(("dx", "dw", "db"), got):
        tr.check(g, *ref[name], f"{which} {rows}x{cols} {kind} {name}")


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 33, 200, 256, 257, 264, 511, 1000, 2048, 2049, 4096, 5000, 8184, 8191, 8192, 8193, 8200,
                                  12001, 16384, 20001, 33000, 65536, 65537, 70008])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_backward_widths(which, cols, kind):
    back_case(which, 7, cols, kind, seed=cols)


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 151, 153, 1300, 5000])
@pytest.mark.parametrize("cols", [72, 776])
def test_backward_rows(which, rows, cols):
    back_case(which, rows, cols, "f16", seed=rows)


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dsum,affine", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("cols", [392, 9000, 66000])
def test_backward_forms(which, kind, dsum, affine, cols):
    back_case(which, 33, cols, kind, dsum, affine)


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("cols", [200, 2049, 9001, 66001])
@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_backward_strides(which, pad, offset, cols, kind):
    back_case(which, 40, cols, kind, pad=pad, offset=offset)


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("inplace", ["dout", "dsum"])
@pytest.mark.parametrize("rows,cols", [(2000, 264), (400, 4096), (30, 10000), (700, 333), (200, 9999), (9, 70000)])
def test_backward_in_place(which, inplace, rows, cols):
    back_case(which, rows, cols, "bf16", inplace=inplace)


@pytest.mark.parametrize("which", ["layer", "rms"])
def test_backward_many_rows(which):
    back_case(which, 3000, 8192, "bf16", seed=1)
    back_case(which, 3001, 1003, "bf16", seed=2)
    back_case(which, 700, 16384, "f16", seed=3)
    back_case(which, 301, 30001, "f16", seed=4)
    back_case(which, 2000, 100, "f32", seed=5, pad=1)


def test_backward_of_nothing():
    x, dw, db = torch.zeros((0, 50), device="cuda"), torch.full((50,), 7.0, device="cuda"), torch.full((50,), 7.0, device="cuda")
    e = torch.zeros(0, device="cuda")
    dx, _, _ = bg.layernorm_backward(x, x, e, e, dweight=dw, dbias=db)
    assert dx.shape == (0, 50) and not dw.any() and not db.any()
    dw.fill_(7)
    assert not bg.rmsnorm_backward(x, x, dweight=dw)[1].any()


def test_backward_repeats_itself():
    """Sums over rows come in one order: the same bits each time."""
    x, d = rand((2500, 1000), 1).half(), rand((2500, 1000), 2).half()
    first = bg.rmsnorm_backward(d, x)
    for _ in range(3):
        again = bg.rmsnorm_backward(d, x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_backward_follows_differences():
    """The kernels' gradients along a direction against differences of the 64-bit forward pass."""
    rows, cols = 20, 500
    x, d, v = (rand((rows, cols), i) for i in (1, 2, 3))
    w, b = 1 + 0.2 * rand((cols,), 4), rand((cols,), 5)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    bg.layernorm(x, w, b, mean_out=mean, rstd_out=rstd)
    dx, dw, db = bg.layernorm_backward(d, x, mean, rstd, w)
    step = 1e-6

    def loss(x, w, b):
        return float((tr.layernorm64(x, None, w, b, 1e-5)[0] * d).sum())
    x6, w6, b6, v6, vw = x.double(), w.double(), b.double(), v.double(), rand((cols,), 6).double()
    for got, along, at in ((dx, v6, lambda t: (x6 + t * v6, w6, b6)), (dw, vw, lambda t: (x6, w6 + t * vw, b6)),
                           (db, vw, lambda t: (x6, w6, b6 + t * vw))):
        slope = (loss(*at(step)) - loss(*at(-step))) / (2 * step)
        # a gradient's elements are off by well under 1e-5 of their size, the difference by 1e-8 of the loss's terms
        assert abs(float((got.double() * along).sum()) - slope) < 1e-5 * float((got.double() * along).abs().sum()) + 1e-5
    dx, dw = bg.rmsnorm_backward(d, x, w)

    def rms(x):
        return float((x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w6 * d).sum())
    slope = (rms(x6 + step * v6) - rms(x6 - step * v6)) / (2 * step)
    assert abs(float((dx.double() * v6).sum()) - slope) < 1e-5 * float((dx.double() * v6).abs().sum()) + 1e-5


@pytest.mark.parametrize("which", ["layer", "rms"])
@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_backward_at_the_matrix_ends(which, kind):
    """Rows off the grid in tensors of their own size: nothing before the first element or behind the last is there."""
    for rows, cols in ((3, 77), (2, 1001), (5, 8195)):
        back_case(which, rows, cols, kind, pad=0, offset=0)
        x = rand((rows * cols + 5,), 1).to(TD[kind])[3: 3 + rows * cols].view(rows, cols)
        d = rand((rows * cols + 1,), 2).to(TD[kind])[1:].view(rows, cols)
        got = bg.rmsnorm_backward(d, x)
        ref = tr.rmsnorm_backward64(d, x, None, 1e-6, None)
        tr.check(got[0], *ref["dx"], "dx")
        tr.check(got[1], *ref["dw"], "dw")


def test_backward_in_a_graph():
    """Captured calls share a workspace of the graph's pool and replay with new inputs."""
    x, d = rand((600, 1000), 1).bfloat16(), rand((600, 1000), 2).bfloat16()
    dx, dw = torch.empty_like(x), torch.empty(1000, device="cuda")
    bg.rmsnorm_backward(d, x, dx=dx, dweight=dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.rmsnorm_backward(d, x, dx=dx, dweight=dw)
    x.copy_(rand((600, 1000), 3))
    graph.replay()
    torch.cuda.synchronize()
    ref = tr.rmsnorm_backward64(d, x, None, 1e-6, None)
    tr.check(dx, *ref["dx"], "dx")
    tr.check(dw, *ref["dw"], "dw")
