"""Sums over more tokens, channels or elements than one tensor-core accumulator takes, of terms of one sign, where that
accumulator's cutting short adds up: no accumulator sums more than 32768 products (512 where a gated layer's K is longer),
and their sums are added in fp32."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

LONGEST = 32768


def positive(rows, cols, seed, kind):
    """Uniform in [0, 1), filled piece by piece."""
    gen = torch.Generator("cuda").manual_seed(seed)
    t = torch.empty((rows, cols), dtype=kind, device="cuda")
    for i in range(0, rows, 32768):
        t[i: i + 32768] = torch.rand(t[i: i + 32768].shape, generator=gen, device="cuda")
    return t


def check(got, ref, length, pieces, what):
    """ref: a sum of positive products, so its own sum of magnitudes."""
    tr.check(got, ref, tr.product_error(length, ref) + pieces * tr.U * ref, what)


def quiet():
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_many_tokens(kind):
    """dw over 400 001 tokens; 2560 x 2048 fill the machine without shares."""
    M, N, K = 400_001, 2560, 2048
    d, x = positive(M, N, 1, kind), positive(M, K, 2, kind)
    d *= 2.0 ** -8
    w = torch.zeros((N, K), dtype=kind, device="cuda")
    db = torch.empty(N, device="cuda")
    dx, dw = bg.matmul_backward(d, x, w, dbias=db)
    quiet()
    for at in (slice(0, 64), slice(N - 64, N)):
        check(dw[at, :256], d[:, at].double().T @ x[:, :256].double(), LONGEST, 13, "dw")
        assert bool(((db[at].double() - d[:, at].double().sum(0)).abs() <= tr.column_adds(M) * tr.U * db[at].double()).all())
    assert not dx[::1000].any()


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_many_channels(kind):
    """dx over 300 008 channels."""
    M, N, K = 2560, 300_008, 2048
    d, w = positive(M, N, 1, kind), positive(N, K, 2, kind)
    d *= 2.0 ** -8
    x = torch.zeros((M, K), dtype=kind, device="cuda")
    dx, dw = bg.matmul_backward(d, x, w)
    quiet()
    for at in (slice(0, 64), slice(M - 64, M)):
        check(dx[at, :256], d[at].double() @ w[:, :256].double(), LONGEST, 10, "dx")
    assert not dw[::1000].any()


def test_gated_gradients():
    """dx over 2 x 160 000 channels and dw over 140 000 tokens; dg = dout u and du = dout g are exact, dout a power of two."""
    kind = torch.float16
    M, N, K = 2304, 160_000, 2048
    x, wg, wu = torch.zeros((M, K), dtype=kind, device="cuda"), positive(N, K, 1, kind), positive(N, K, 2, kind)
    g, u = positive(M, N, 3, kind), positive(M, N, 4, kind)
    d = torch.full((M, N), 2.0 ** -8, dtype=kind, device="cuda")
    dx, _, _ = bg.matmul_gated_backward(d, x, wg, wu, g, u, act=bg.ACT_NONE)
    quiet()
    ref = (u[:64].double() @ wg[:, :256].double() + g[:64].double() @ wu[:, :256].double()) * 2.0 ** -8
    # u and g times 2^-8 are exact in f16 but below 2^-14, by half a step of 2^-24 each
    lost = 2.0 ** -25 * (wg[:, :256].double().sum(0) + wu[:, :256].double().sum(0))
    tr.check(dx[:64, :256], ref, tr.product_error(LONGEST, ref) + 10 * tr.U * ref + lost, "dx")
    del wg, wu, g, u, d, x, dx
    M, N, K = 140_000, 1280, 2048
    x, wg = positive(M, K, 1, kind), torch.zeros((N, K), dtype=kind, device="cuda")
    g, u = positive(M, N, 3, kind), positive(M, N, 4, kind)
    d = torch.full((M, N), 2.0 ** -8, dtype=kind, device="cuda")
    _, dwg, dwu = bg.matmul_gated_backward(d, x, wg, wg, g, u, act=bg.ACT_NONE)
    quiet()
    lost = 2.0 ** -25 * x[:, :256].double().sum(0)
    for got, of in ((dwg, u), (dwu, g)):
        ref = of[:, :64].double().T @ x[:, :256].double() * 2.0 ** -8
        tr.check(got[:64, :256], ref, tr.product_error(LONGEST, ref) + 5 * tr.U * ref + lost, "dw")


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 16, 50, 300])
@pytest.mark.parametrize("K", [32769, 262_144])
def test_gated_long_rows(kind, M, K):
    """A gated layer over K channels in, summed in pieces of 512; 10 240 channels out leave no clusters."""
    N = 10_240 if M == 16 else 200
    x, wg, wu = positive(M, K, 1, kind), positive(N, K, 2, kind), positive(N, K, 3, kind)
    x *= 2.0 ** -8
    g, u = torch.empty((M, N), dtype=kind, device="cuda"), torch.empty((M, N), dtype=kind, device="cuda")
    wu *= 2.0 ** -6
    y = bg.matmul_gated(x, wg, wu, act=bg.ACT_NONE, gate_out=g, up_out=u)
    quiet()
    x6, pieces = x.double(), K / 512 + 8
    both = [x6 @ w[:200].double().T for w in (wg, wu)]
    for got, ref in zip((g, u), both):
        check(got[:, :200], ref, 512, pieces, "sums")
    e = [tr.product_error(512, r) + pieces * tr.U * r for r in both]
    tr.check(y[:, :200], both[0] * both[1], e[0] * both[1] + e[1] * both[0] + e[0] * e[1] + 2 * tr.U * both[0] * both[1], "out")
