"""The 64-bit gradients that the GPU tests compare with, against differences and torch's autograd in 64 bits, without a
GPU."""
import pytest
import torch

from tests import train_ref as tr


def rand(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("weight", [False, True])
def test_layernorm_gradients(weight):
    x, d, s = (rand(5, 33, seed=i) for i in (1, 2, 3))
    w, b = (rand(33, seed=4), rand(33, seed=5)) if weight else (None, None)
    leaves = [t.clone().requires_grad_() for t in ((x, w, b) if weight else (x,))]
    y = torch.nn.functional.layer_norm(leaves[0], (33,), *(leaves[1:] if weight else (None, None)), eps=1e-5)
    assert torch.allclose(tr.layernorm64(x, None, w, b, 1e-5)[0], y.detach(), rtol=1e-12, atol=1e-13)
    want = torch.autograd.grad((y * d).sum() + (leaves[0] * s).sum(), leaves)
    _, _, _, m, _, r, _ = tr.layernorm64(x, None, w, b, 1e-5)
    got = tr.layernorm_backward64(d, x, m, r, w, s)
    for name, g in zip(("dx", "dw", "db"), want):
        assert torch.allclose(got[name][0], g, rtol=1e-10, atol=1e-12), name


@pytest.mark.parametrize("weight", [False, True])
def test_rmsnorm_gradients(weight):
    x, d = rand(4, 21, seed=1), rand(4, 21, seed=2)
    w = rand(21, seed=3) if weight else None

    def loss(x, w):
        return (d * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (1 if w is None else w)).sum()
    got = tr.rmsnorm_backward64(d, x, w, 1e-6, None)
    v, step = rand(4, 21, seed=5), 1e-5
    slope = float(loss(x + step * v, w) - loss(x - step * v, w)) / (2 * step)
    assert abs(slope - float((got["dx"][0] * v).sum())) < 1e-8 * (1 + abs(slope))
    if weight:
        v = rand(21, seed=6)
        slope = float(loss(x, w + step * v) - loss(x, w - step * v)) / (2 * step)
        assert abs(slope - float((got["dw"][0] * v).sum())) < 1e-8 * (1 + abs(slope))


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu", "none"])
def test_activation_slopes(kind):
    z = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    z = z[z.abs() > 1e-3]
    step = 1e-5
    want = (tr.act64(kind, z + step)[0] - tr.act64(kind, z - step)[0]) / (2 * step)
    assert torch.allclose(tr.act64(kind, z)[1], want, rtol=1e-8, atol=1e-9)
