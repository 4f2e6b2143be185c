"""The products' kernels and cuts one by one, each with more than one of whatever it walks over: the pairs' tiles of 256
channels with more tiles than pairs and several pieces of K, and tiles of 16 to 128 tokens whose K one to eight CTAs
share.  The sizes choose what the names say on 152 SMs."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref_gpu as lr

pytestmark = pytest.mark.gpu

TD, rand = lr.TD, lr.rand


def case(M, N, K, kind, out, act="none", combine="none", bias=True, other_kind=None, pad=0, in_place=False, seed=1):
    mx = kind == "mx"
    if mx:
        xq, wq = bg.mx_quantize(rand((M, K), seed)), bg.mx_quantize(rand((N, K), seed + 1, K ** -0.5))
        x, w = lr.decoded(*xq), lr.decoded(*wq)
    else:
        xs, ws = lr.strided(rand((M, K), seed), pad, TD[kind]), lr.strided(rand((N, K), seed + 1, K ** -0.5), pad, TD[kind])
        x, w = xs.double(), ws.double()
    b = rand((N,), seed + 2) if bias else None
    side = TD[other_kind or ("bf16" if out == "mx" else out)]
    other = lr.strided(rand((M, N), seed + 3), pad, side) if combine != "none" else None
    o64 = other.double() if other is not None else None
    y = other if in_place else lr.strided(torch.zeros((M, N), device="cuda"), pad, TD[out])
    if not in_place and out != "mx":
        y.fill_(float("nan"))
    kw = {"act": bg.ACT_NAMES[act], "other": other, "combine": bg.COMBINE_NAMES[combine], "out": y}
    got = bg.matmul_mx(*xq, *wq, b, **kw) if mx else bg.matmul(xs, ws, b, **kw)
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0
    ref, d = lr.product64(x, w, b, act, o64, combine, out in ("f32", "mx"), mx)
    what = f"{M}x{N}x{K} {kind}->{out} {act} {combine}"
    if out == "mx":
        lr.check_mx(*got, ref, d, what)
        return
    assert got is y
    lr.check_float(y, ref, d, what)
    if out == "f32":
        off = 4 * 2.0 ** -24 if mx else 32 * 2.0 ** -23 * 0.5 ** 0.5 + (K / 512 + 8) ** 0.5 * 2.0 ** -24
        if act == "none" and combine != "mul":      # the sum itself, and roundings of no more than its size
            assert float((y.double() - ref).norm() / ref.norm()) <= off + 2 * 2.0 ** -24, what
    if pad:
        assert torch.isnan(y._base[:, N:]).all(), f"{what}: written past the row"


# 99, 85 (ragged in every way), 170 and 158 tiles on 76 pairs
WIDE = [(2050, 2568, 2600), (1300, 4104, 1000), (2560, 4104, 2600), (20000, 260, 300)]


@pytest.mark.parametrize("M,N,K", WIDE)
@pytest.mark.parametrize("kind,out,act,combine", [
    ("bf16", "bf16", "gelu_tanh", "none"), ("f16", "f16", "silu", "mul"), ("f16", "f32", "none", "add"), ("bf16", "f32", "none", "none"),
    ("mx", "bf16", "none", "add"), ("mx", "f16", "gelu", "none"), ("mx", "f32", "none", "add"), ("mx", "mx", "gelu", "none"),
    ("mx", "mx", "silu", "mul")])
def test_tiles_of_256_channels(M, N, K, kind, out, act, combine):
    case(M, N, K, kind, out, act, combine)


@pytest.mark.parametrize("N", [5001, 2570])
@pytest.mark.parametrize("kind,out,act,combine,other", [
    ("bf16", "bf16", "silu", "mul", None), ("f16", "f32", "none", "add", None), ("f16", "f16", "relu", "add", "f32"),
    ("mx", "f16", "none", "none", None), ("mx", "f32", "none", "add", None), ("mx", "mx", "gelu", "add", "f32")])
def test_tiles_of_256_channels_off_the_grid(N, kind, out, act, combine, other):
    case(2100 if N == 2570 else 1537, N, 1000, kind, out, act, combine, other_kind=other, pad=3)


@pytest.mark.parametrize("kind,out,other", [("bf16", "bf16", "f32"), ("f16", "f16", "bf16"), ("f16", "f32", "f16"), ("mx", "bf16", "f16"),
                                            ("mx", "mx", "f32"), ("mx", "mx", "f16")])
def test_other_of_another_type(kind, out, other):
    case(2050, 2568, 520, kind, out, "relu", "mul", other_kind=other)


@pytest.mark.parametrize("M,N", [(2050, 2568), (1537, 5001), (300, 1000)])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32"), ("mx", "f16"), ("mx", "f32")])
@pytest.mark.parametrize("combine", ["add", "mul"])
def test_other_is_the_output(M, N, kind, out, combine):
    case(M, N, 520, kind, out, "none", combine, in_place=True)


@pytest.mark.parametrize("M,N,K", [(2500, 2600, 8192), (1100, 6000, 4112)])
@pytest.mark.parametrize("kind,out", [("f16", "bf16"), ("bf16", "f32"), ("mx", "bf16"), ("mx", "f32"), ("mx", "mx")])
def test_long_sums(M, N, K, kind, out):
    case(M, N, K, "bf16" if (kind, out) == ("f16", "bf16") else kind, out, "none", "add")


# 128, 64, 32 and 16 tokens to a tile, K of a tile shared by so many CTAs
FEW = {
    "128 in 2": (300, 5000, 8192), "128 in 2 alone": (500, 2000, 4096), "128 in 3": (200, 5000, 4096), "128 in 3 alone": (100, 5000, 4096),
    "128 in 4 alone": (200, 2000, 4096), "64 in 2 alone": (200, 2000, 2048), "64 in 3": (100, 5000, 1024), "64 in 3 alone": (33, 5000, 2048),
    "64 in 4 alone": (100, 2000, 2048), "64 in 8 alone": (33, 2000, 8192), "32 in 1": (128, 5000, 256), "32 in 3": (20, 5000, 1024),
    "32 in 4": (20, 5000, 8192), "32 in 8": (20, 2000, 4096), "16 in 2": (33, 5000, 1024), "16 in 3": (1, 5000, 1024),
    "16 in 8": (1, 100, 2048)}


@pytest.mark.parametrize("cut", FEW)
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32")])
def test_few_tokens(cut, kind, out):
    case(*FEW[cut], kind, out, "gelu", "add")


FEW_MX = {
    "128 in 2": (300, 5000, 4096), "128 in 2 alone": (500, 2000, 8192), "128 in 3": (200, 5000, 4096), "128 in 3 alone": (100, 5000, 8192),
    "128 in 4 alone": (200, 2000, 8192), "64 in 1 alone": (33, 100, 256), "64 in 2": (100, 5000, 1024), "64 in 3": (100, 5000, 2048),
    "64 in 3 alone": (33, 5000, 2048), "64 in 8 alone": (33, 100, 4096), "32 in 3": (20, 5000, 2048), "32 in 8": (20, 100, 4096),
    "16 in 3": (1, 5000, 2048), "16 in 8": (1, 100, 4096)}


@pytest.mark.parametrize("cut", FEW_MX)
@pytest.mark.parametrize("out", ["f16", "f32", "mx"])
def test_few_tokens_mx(cut, out):
    case(*FEW_MX[cut], "mx", out, "silu", "mul")


@pytest.mark.parametrize("kind", ["f16", "mx"])
def test_nan_and_infinity_stay_in_their_rows(kind):
    M, N, K = 2050, 2568, 520
    x, w = rand((M, K), 1), rand((N, K), 2, K ** -0.5)
    if kind == "f16":
        x, w = x.half(), w.half()
        call = lambda: bg.matmul(x, w)     # noqa: E731
        clean = call()
        x[700, 5], x[1500, 519] = float("nan"), float("inf")
    else:
        (q, s), (p, t) = bg.mx_quantize(x), bg.mx_quantize(w)
        call = lambda: bg.matmul_mx(q, s, p, t)    # noqa: E731
        clean = call()
        x[700, 5], x[1500, 519] = float("nan"), float("inf")
        bg.mx_quantize(x, out=q, scale=s)
    got = call()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[700, 1500]] = False
    assert torch.isnan(got[700]).all() and not torch.isfinite(got[1500]).any() and torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32"), ("mx", "mx")])
def test_same_bits_every_time(kind, out):
    M, N, K = 2560, 4104, 2600
    if kind == "mx":
        a, b = bg.mx_quantize(rand((M, K), 1)), bg.mx_quantize(rand((N, K), 2, K ** -0.5))
        call = lambda: torch.cat([t.view(torch.uint8).reshape(-1) for t in bg.matmul_mx(*a, *b, out_dtype=TD[out])])    # noqa: E731
    else:
        a, b = rand((M, K), 1).to(TD[kind]), rand((N, K), 2, K ** -0.5).to(TD[kind])
        call = lambda: bg.matmul(a, b, out_dtype=TD[out])    # noqa: E731
    first = call()
    for _ in range(10):
        assert torch.equal(call(), first)
