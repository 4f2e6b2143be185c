"""gelu against 64 bits with a relative bound, for negative z as well, where its values are small.

z Phi(z) = z t P(t) exp(-z^2 / 2): the exponent z^2 log2(e) / 2 is rounded twice, by 2^-24 of itself each, which is z^2 2^-24
of the value; the power and the reciprocal are off by 2 and 1 units of 2^-23, the fit by 2^-23, and eight products and
sums by 2^-24 each: (z^2 + 16) 2^-24, half as much again allowed for.  Then the output's rounding."""
import numpy as np
import pytest
import torch
from scipy.special import log_ndtr

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref as lr

pytestmark = pytest.mark.gpu


def zs():
    """Every 16-bit float from -12 to 8 of at least 2^-8."""
    z = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.uint16).view(torch.float16)
    return z[(z >= -12) & (z <= 8) & (z.abs() >= 2.0 ** -8)]


@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("many", [False, True])
def test_relative_to_the_value(out, many):
    z = zs()
    x, w = z[:, None].cuda(), torch.ones(1, 1).half().cuda()
    if not many:
        x, w = w, x                   # one token, a channel for each z
    y = bg.matmul(x, w, act=bg.ACT_GELU, out_dtype=out).reshape(-1).cpu().double().numpy()
    z = z.double().numpy()
    ref = z * np.exp(log_ndtr(z))
    bound = np.abs(ref) * (z * z + 16) * 1.5 * 2.0 ** -24
    bound = bound + lr.U[out] * (np.abs(ref) + bound) + lr.TINY[out]
    err = np.abs(y - ref)
    assert (err <= bound).all(), f"worst {np.max(err / bound):.2f} of the bound, at z = {z[np.argmax(err / bound)]}"


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("many", [False, True])
def test_quotients_relative_to_the_value(act, out, many):
    """z / (1 + exp(-v)), v = z or 2 sqrt(2/pi) (z + 0.044715 z^3): v's value and its product with log2(e) are off by at most
    5 times 2^-24 of v, so the power by 5 |v| 2^-24; the power, sum, reciprocal and product by 8 times 2^-24 together.  Where
    1 + exp(-v) passes 2^126 its reciprocal is flushed to zero: 16 * 2^-126."""
    z = zs()
    x, w = z[:, None].cuda(), torch.ones(1, 1).half().cuda()
    if not many:
        x, w = w, x
    y = bg.matmul(x, w, act=bg.ACT_NAMES[act], out_dtype=out).reshape(-1).cpu().double().numpy()
    z = z.double().numpy()
    v = z if act == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    ref = z / (1 + np.exp(-v))
    bound = np.abs(ref) * (5 * np.abs(v) + 8) * 2.0 ** -24 + 2.0 ** -122
    bound = bound + lr.U[out] * (np.abs(ref) + bound) + lr.TINY[out]
    err = np.abs(y - ref)
    assert (err <= bound).all(), f"worst {np.max(err / bound):.2f} of the bound, at z = {z[np.argmax(err / bound)]}"
