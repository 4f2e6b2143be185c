"""How exactly the products sum: 32-bit and MXFP8 outputs hold K in pieces.

Bounds on the error's 2-norm over the result's, against 64 bits.
MXFP8 operands: four of fp32's half steps (2^-24 each), which a plain fp32 product of these sizes keeps too.
16-bit operands: a piece is 32 additions into the tensor core's accumulator, each cut short by at most 2^-23 of the
partial sum; the partial sums' root mean square over the piece is sqrt(1/2) of the whole's, and the pieces' errors add
up like the pieces do.  Then the fp32 additions of K / 512 pieces and 8 shares, each off by 2^-24 of a partial sum.
One sum over all of K = 16384 is off by 512 such cuts, of which half (1.5e-5) or more are seen."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

MX = torch.float8_e4m3fn


def rand(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale


def decoded(q, scale):
    """An MXFP8 matrix in 64 bits, on the GPU."""
    rows, cols = q.shape
    a, b = -(-rows // 128), -(-cols // 128)
    code = scale.view(torch.uint8).reshape(a, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(a * 128, b * 4)[:rows]
    return q.double() * torch.pow(2.0, code.double() - 127).repeat_interleave(32, 1)[:, :cols]


def off(y, ref):
    return float((y.double() - ref).norm() / ref.norm())


SIZES = [(1, 256), (40, 512), (100, 384), (300, 1000), (1024, 2048)]


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("K", [8192, 16384])
def test_mx_sums(M, N, K):
    x, xs = bg.mx_quantize(rand((M, K), 1))
    w, ws = bg.mx_quantize(rand((N, K), 2, K ** -0.5))
    y = bg.matmul_mx(x, xs, w, ws, out_dtype=torch.float32)
    assert off(y, decoded(x, xs) @ decoded(w, ws).T) <= 4 * 2.0 ** -24


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_16_bit_sums(M, N, dtype):
    K = 16384
    x, w = rand((M, K), 3).to(dtype), rand((N, K), 4, K ** -0.5).to(dtype)
    y = bg.matmul(x, w, out_dtype=torch.float32)
    assert off(y, x.double() @ w.double().T) <= 32 * 2.0 ** -23 * 0.5 ** 0.5 + (K / 512 + 8) ** 0.5 * 2.0 ** -24


@pytest.mark.parametrize("K", [320, 2048, 2080, 4112, 16384])
@pytest.mark.parametrize("M,N", [(1, 256), (40, 208), (100, 96), (260, 512), (300, 1008), (1300, 2560)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_mx_output_is_the_32_bit_one_quantised(M, N, K, act):
    """An MXFP8 output is summed as exactly as a 32-bit one, however long K is: the same bits after rounding."""
    x, xs = bg.mx_quantize(rand((M, K), K + M))
    w, ws = bg.mx_quantize(rand((N, K), K + M + 1, K ** -0.5))
    b = rand((N,), 3)
    q, s = bg.matmul_mx(x, xs, w, ws, b, act=bg.ACT_NAMES[act], out_dtype=MX)
    y = bg.matmul_mx(x, xs, w, ws, b, act=bg.ACT_NAMES[act], out_dtype=torch.float32)
    q2, s2 = bg.mx_quantize(y)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s.view(torch.uint8), s2.view(torch.uint8))
    assert bg.bigemm_last_device_error() == 0
