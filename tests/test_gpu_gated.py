"""GPU parity of a gated layer's products and of the products' gradients against their 64-bit definitions (train_ref has
the bounds)."""
import math

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16}


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def strided(t, pad, dtype, offset=0):
    """The matrix as columns of a wider tensor, NaN in the others."""
    big = torch.full((t.shape[0], t.shape[1] + pad + offset), float("nan"), device="cuda").to(dtype)
    big[:, offset: offset + t.shape[1]] = t.to(dtype)
    return big[:, offset: offset + t.shape[1]]


def empty(rows, cols, pad, dtype, offset=0):
    """An output among NaN, with a row behind its last."""
    big = torch.full((rows + 1, cols + pad + offset), float("nan"), device="cuda").to(dtype)
    return big[:rows, offset: offset + cols]


def untouched(t):
    base, rows, cols, offset = t._base, t.shape[0], t.shape[1], t.storage_offset()
    return bool(torch.isnan(base[rows:]).all() and torch.isnan(base[:, :offset]).all() and torch.isnan(base[:, offset + cols:]).all())


def quiet():
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0


def gated_case(M, N, K, kind="bf16", act="silu", bias=False, keep=True, pad=0, offset=0, seed=1):
    x = strided(rand((M, K), seed), pad, TD[kind], offset)
    wg, wu = (strided(rand((N, K), seed + i) / math.sqrt(K), pad, TD[kind], offset) for i in (1, 2))
    b, c = (rand((N,), seed + 3), rand((N,), seed + 4)) if bias else (None, None)
    y = empty(M, N, pad, TD[kind], offset)
    g, u = (empty(M, N, pad, TD[kind], offset) for _ in range(2)) if keep else (None, None)
    got = bg.matmul_gated(x, wg, wu, b, c, act=bg.ACT_NAMES[act], out=y, gate_out=g, up_out=u)
    quiet()
    assert got is y
    ref = tr.gated64(x, wg, wu, b, c, act)
    for name, t in (("y", y), ("g", g), ("u", u)):
        if t is not None:
            what = f"{M}x{N}x{K} {kind} {act} {name}"
            tr.check(t, *ref[name], what)
            tr.check_norm(t, ref[name][0], 1, what)
            assert untouched(t), what


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("N,K", [(64, 64), (200, 520), (1024, 1024)])
def test_gated_tokens(M, N, K):
    gated_case(M, N, K, seed=M)


@pytest.mark.parametrize("N", [1, 7, 8, 31, 32, 63, 65, 127, 129, 1000, 5001])
@pytest.mark.parametrize("M", [3, 300])
def test_gated_channels(M, N):
    gated_case(M, N, 200, "f16", bias=True, seed=N)


@pytest.mark.parametrize("K", [1, 2, 8, 15, 64, 72, 1000, 1001, 4096, 9000])
@pytest.mark.parametrize("M", [1, 40, 400])
def test_gated_lengths(M, K):
    gated_case(M, 264, K, seed=K)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M,keep,bias", [(5, False, False), (5, True, True), (700, False, True), (700, True, False)])
def test_gated_forms(act, kind, M, keep, bias):
    gated_case(M, 712, 384, kind, act, bias, keep)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("M", [9, 520])
def test_gated_strides(M, pad, offset):
    gated_case(M, 328, 264, "f16", "gelu", True, pad=pad, offset=offset)


def test_gated_many_tiles():
    """More tiles than pairs, ragged in every axis."""
    gated_case(3000, 2500, 328, "bf16", keep=True)
    gated_case(300, 20000, 72, "f16", keep=False)


def test_gated_kept_singly():
    x, wg, wu = rand((300, 128), 1).bfloat16(), rand((256, 128), 2).bfloat16(), rand((256, 128), 3).bfloat16()
    for M in (4, 300):
        g, u, g1, u1 = (torch.empty((M, 256), dtype=torch.bfloat16, device="cuda") for _ in range(4))
        y = bg.matmul_gated(x[:M], wg, wu, gate_out=g, up_out=u)
        a, b = bg.matmul_gated(x[:M], wg, wu, gate_out=g1), bg.matmul_gated(x[:M], wg, wu, up_out=u1)
        assert torch.equal(y, a) and torch.equal(y, b) and torch.equal(g, g1) and torch.equal(u, u1)
        assert torch.equal(y, bg.matmul_gated(x[:M], wg, wu))
    assert bg.matmul_gated(x[:0], wg, wu).shape == (0, 256)


def test_gated_nan_stays_in_its_token():
    wg, wu = rand((300, 128), 2).half(), rand((300, 128), 3).half()
    for M in (6, 300):
        x = rand((M, 128), 1).half()
        clean = bg.matmul_gated(x, wg, wu)
        x[2, 5] = float("nan")
        got = bg.matmul_gated(x, wg, wu)
        keep = [i for i in range(M) if i != 2]
        assert torch.isnan(got[2]).all() and torch.equal(got[keep], clean[keep])


# --------------------------------------------------------------------- gradients of a product

def linear_case(M, N, K, kind="bf16", bias=True, pad=0, offset=0, seed=1):
    d, x = strided(rand((M, N), seed) * 0.1, pad, TD[kind], offset), strided(rand((M, K), seed + 1), pad, TD[kind], offset)
    w = strided(rand((N, K), seed + 2) / math.sqrt(K), pad, TD[kind], offset)
    dx, dw = empty(M, K, pad, TD[kind], offset), empty(N, K, pad, TD[kind], offset)
    db = torch.full((N,), float("nan"), device="cuda") if bias else None
    got = bg.matmul_backward(d, x, w, dx=dx, dw=dw, dbias=db)
    quiet()
    assert got[0] is dx and got[1] is dw
    ref = tr.product_backward64(d, x, w)
    for name, t in (("dx", dx), ("dw", dw), ("db", db)):
        if t is not None:
            what = f"{M}x{N}x{K} {kind} {name}"
            tr.check(t, *ref[name], what)
            if name != "db":
                tr.check_norm(t, ref[name][0], 1, what)
                assert untouched(t), what


@pytest.mark.parametrize("M", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("N,K", [(64, 64), (328, 200), (1024, 1024)])
def test_linear_backward_tokens(M, N, K):
    linear_case(M, N, K, seed=M)


@pytest.mark.parametrize("N", [1, 7, 8, 32, 63, 65, 129, 255, 257, 1000, 5001])
@pytest.mark.parametrize("M", [3, 300])
def test_linear_backward_outputs(M, N):
    linear_case(M, N, 136, "f16", seed=N)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 24, 31, 32, 33, 63, 65, 129, 255, 256, 257, 1000, 5001])
@pytest.mark.parametrize("M,N", [(3, 520), (300, 72)])
def test_linear_backward_inputs(M, N, K):
    linear_case(M, N, K, seed=K)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M", [9, 520])
def test_linear_backward_strides(M, pad, offset, kind):
    linear_case(M, 328, 264, kind, pad=pad, offset=offset)


def test_linear_backward_shares():
    """Few tokens and many outputs: dx's units are cut along the summed axis."""
    for M, N, K in ((1, 16384, 256), (5, 9001, 1000), (100, 4096, 4096), (257, 8192, 512), (40, 16384, 37)):
        linear_case(M, N, K, seed=M, bias=False)


def test_linear_backward_shares_of_dw():
    """Many tokens and few outputs: dw's units are cut along the tokens, alone and with dx's."""
    for M, N, K in ((3296, 73, 288), (9000, 16, 40), (5000, 200, 513), (4096, 128, 2048), (1500, 700, 90)):
        linear_case(M, N, K, seed=M)
    linear_case(6000, 100, 264, "f16", pad=1)


def test_gated_backward_shares_of_dw():
    back_case(4608, 176, 320, "f16", "none")
    back_case(5730, 90, 129, "bf16", "silu")


@pytest.mark.parametrize("M", [1, 31, 33, 255])
@pytest.mark.parametrize("N,K", [(40, 1), (31, 63), (65, 65), (100, 127), (300, 1025)])
def test_linear_backward_off_the_grid(M, N, K):
    """Odd rows of outputs, whole matrices and columns of wider ones."""
    linear_case(M, N, K, "bf16", pad=0, seed=K)
    linear_case(M, N, K, "f16", pad=3, offset=1, seed=K)
    gated_case(M, N, K, "bf16", pad=0, seed=K)
    gated_case(M, K, N, "f16", pad=1, offset=1, seed=K)


def test_linear_backward_many_units():
    linear_case(3000, 2500, 1800, "bf16")
    linear_case(5000, 72, 2064, "f16")


def test_linear_backward_of_nothing():
    x, w = torch.zeros((0, 24), dtype=torch.float16, device="cuda"), rand((16, 24), 1).half()
    d = torch.zeros((0, 16), dtype=torch.float16, device="cuda")
    dw, db = empty(16, 24, 5, torch.float16), torch.full((16,), 7.0, device="cuda")
    dx, _ = bg.matmul_backward(d, x, w, dw=dw, dbias=db)
    quiet()
    assert dx.shape == (0, 24) and not dw.any() and not db.any() and untouched(dw)


def test_linear_backward_nan_stays_in_its_place():
    d, x, w = rand((300, 200), 1).half(), rand((300, 136), 2).half(), rand((200, 136), 3).half()
    cx, cw = bg.matmul_backward(d, x, w)
    d[7, 11] = float("nan")
    db = torch.empty(200, device="cuda")
    dx, dw = bg.matmul_backward(d, x, w, dbias=db)
    rows, chans = [i for i in range(300) if i != 7], [i for i in range(200) if i != 11]
    assert torch.isnan(dx[7]).all() and torch.equal(dx[rows], cx[rows])
    assert torch.isnan(dw[11]).all() and torch.equal(dw[chans], cw[chans])
    assert torch.isnan(db[11]) and torch.isfinite(db[chans]).all()


# --------------------------------------------------------------------- gradients of a gated layer

def back_case(M, N, K, kind="bf16", act="silu", bias=True, pad=0, offset=0, seed=1):
    d, x = strided(rand((M, N), seed) * 0.1, pad, TD[kind], offset), strided(rand((M, K), seed + 1), pad, TD[kind], offset)
    wg, wu = (strided(rand((N, K), seed + i) / math.sqrt(K), pad, TD[kind], offset) for i in (2, 3))
    g, u = (strided(rand((M, N), seed + i), pad, TD[kind], offset) for i in (4, 5))
    dx = empty(M, K, pad, TD[kind], offset)
    dwg, dwu = (empty(N, K, pad, TD[kind], offset) for _ in range(2))
    dbg, dbu = (torch.full((N,), float("nan"), device="cuda") for _ in range(2)) if bias else (None, None)
    got = bg.matmul_gated_backward(d, x, wg, wu, g, u, act=bg.ACT_NAMES[act], dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=dbg,
                                   dbias_up=dbu)
    quiet()
    assert got[0] is dx and got[1] is dwg and got[2] is dwu
    ref = tr.gated_backward64(d, x, wg, wu, g, u, act)
    for name, t in (("dx", dx), ("dwg", dwg), ("dwu", dwu), ("dbg", dbg), ("dbu", dbu)):
        if t is not None:
            what = f"{M}x{N}x{K} {kind} {act} {name}"
            tr.check(t, *ref[name], what)
            if not name.startswith("db"):
                tr.check_norm(t, ref[name][0], 2, what)
                assert untouched(t), what


@pytest.mark.parametrize("M", [1, 2, 31, 64, 65, 128, 129, 257, 700])
@pytest.mark.parametrize("N,K", [(64, 64), (328, 200), (1024, 512)])
def test_gated_backward_tokens(M, N, K):
    back_case(M, N, K, seed=M)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 65, 129, 257, 1000, 5001])
@pytest.mark.parametrize("M", [3, 300])
def test_gated_backward_channels(M, N):
    back_case(M, N, 136, "f16", seed=N)


@pytest.mark.parametrize("K", [1, 7, 8, 33, 64, 129, 257, 1000, 3001])
@pytest.mark.parametrize("M,N", [(3, 520), (300, 72)])
def test_gated_backward_inputs(M, N, K):
    back_case(M, N, K, seed=K)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
def test_gated_backward_forms(act, kind, bias):
    back_case(200, 392, 264, kind, act, bias)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("M", [9, 520])
def test_gated_backward_strides(M, pad, offset):
    back_case(M, 328, 264, "f16", "gelu", pad=pad, offset=offset)


def test_gated_backward_many_units():
    back_case(1500, 2500, 1800, "bf16")
    back_case(20, 16384, 264, "f16")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_over_every_float(act):
    """A single token's bias gradients are the activation and its slope, unrounded: over every bf16 from -30 to 30 and over
    large ones, where they must be finite."""
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = bits[torch.isfinite(bits) & (bits.float().abs() >= 2.0 ** -126)].cuda()[None]
    N = z.shape[1]
    one = torch.ones((1, N), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((N, 8), dtype=torch.bfloat16, device="cuda")
    s, a = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    bg.matmul_gated_backward(one, torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda"), w, w, z, one, act=bg.ACT_NAMES[act],
                             dbias_gate=s, dbias_up=a)
    quiet()
    assert torch.isfinite(s).all() and torch.isfinite(a).all()
    va, vs = tr.act64(act, z[0].double())
    near = z[0].abs() <= 30
    z6 = z[0].double()
    for got, want, size in ((a, va, z6.abs().clamp(min=1)), (s, vs, torch.ones_like(z6))):
        err = (got.double() - want).abs()
        assert float((err / size)[near].max()) <= 2.0 ** -19
    # far out the slopes and quotients are exactly 0 and 1
    far = z6.abs() > 30
    assert torch.allclose(s.double()[far], vs[far], rtol=0, atol=1e-9)
    assert torch.allclose(a.double()[far], va[far], rtol=1e-6, atol=1e-9)


def test_gated_backward_of_nothing():
    x, w = torch.zeros((0, 24), dtype=torch.float16, device="cuda"), rand((16, 24), 1).half()
    e = torch.zeros((0, 16), dtype=torch.float16, device="cuda")
    dwg, dwu = (empty(16, 24, 8, torch.float16) for _ in range(2))
    dbg = torch.full((16,), 7.0, device="cuda")
    dx, _, _ = bg.matmul_gated_backward(e, x, w, w, e, e, dw_gate=dwg, dw_up=dwu, dbias_gate=dbg)
    quiet()
    assert dx.shape == (0, 24) and not dwg.any() and not dwu.any() and not dbg.any()


def test_one_bias_gradient_alone():
    M, N, K = 50, 300, 64
    d, x, g, u = (rand(s, i).half() for i, s in enumerate(((M, N), (M, K), (M, N), (M, N))))
    w = rand((N, K), 9).half()
    both = [torch.empty(N, device="cuda") for _ in range(2)]
    bg.matmul_gated_backward(d, x, w, w, g, u, dbias_gate=both[0], dbias_up=both[1])
    one = torch.empty(N, device="cuda")
    bg.matmul_gated_backward(d, x, w, w, g, u, dbias_gate=one)
    assert torch.equal(one, both[0])
    bg.matmul_gated_backward(d, x, w, w, g, u, dbias_up=one)
    quiet()
    assert torch.equal(one, both[1])


def test_backward_repeats_itself():
    """Shares and sums come in one order: the same bits each time."""
    d, x, w = rand((100, 2000), 1).half(), rand((100, 1000), 2).half(), rand((2000, 1000), 3).half()
    first = [torch.empty(2000, device="cuda")]
    first += list(bg.matmul_backward(d, x, w, dbias=first[0]))
    for _ in range(3):
        again = [torch.empty(2000, device="cuda")]
        again += list(bg.matmul_backward(d, x, w, dbias=again[0]))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradients_follow_differences():
    """The gated layer's gradients along directions against differences of the 64-bit forward pass, from what the forward
    call kept: off by the roundings of the kept sums and of the gradients."""
    M, N, K = 60, 200, 96
    x, wg, wu = rand((M, K), 1).half(), (rand((N, K), 2) / 10).half(), (rand((N, K), 3) / 10).half()
    d = (rand((M, N), 4) * 0.1).half()
    g, u = (torch.empty((M, N), dtype=torch.float16, device="cuda") for _ in range(2))
    bg.matmul_gated(x, wg, wu, act=bg.ACT_GELU, gate_out=g, up_out=u)
    grads = bg.matmul_gated_backward(d, x, wg, wu, g, u, act=bg.ACT_GELU)
    quiet()
    at = [t.double() for t in (x, wg, wu)]
    step = 1e-6
    for i, got in enumerate(grads):
        v = rand(got.shape, 5 + i).double()

        def loss(t):
            a = [p + t * v if j == i else p for j, p in enumerate(at)]
            return float((tr.gated64(a[0], a[1], a[2], None, None, "gelu")["y"][0] * d.double()).sum())
        slope = (loss(step) - loss(-step)) / (2 * step)
        # each term of the sum is off by about 2^-11 of its size, four times over, with random signs
        terms = (got.double() * v).norm()
        assert abs(float((got.double() * v).sum()) - slope) < 8 * 2.0 ** -11 * float(terms) + 1e-5
