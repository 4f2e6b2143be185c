"""The calls of a training step of a gated MLP block together (examples/mlp_train.py): its gradients against 64 bits, along
directions, replayed from a graph, and on a stream of its own."""
import os
import sys

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mlp_train  # noqa: E402

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def rand(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def block(tokens, hidden, inner, dtype, layer, seed=1):
    w = mlp_train.weights(hidden, inner, dtype, layer, seed)
    return w, rand((tokens, hidden), seed, dtype), rand((tokens, hidden), seed + 1, dtype), rand((tokens, hidden), seed + 2, dtype)


def check(got, ref, dtype):
    """A gradient passes through at most nine tensors that are rounded to the type (y, gate, up, z, dz, the two sums'
    gradients, dy, itself), each off by up to half a step; their errors are independent, of a third of the square of half a
    step on average, and an activation's slope is at most 1.13, a norm's derivative at most 1 on its rows' scale: in the
    2-norm under sqrt(9 / 3) * 1.13 * 1.13 half steps, and half of that on top for the directions that are longer."""
    most = 1.5 * 3 ** 0.5 * 1.13 ** 2 * HALF[dtype]
    for name, want in ref.items():
        rel = float((got[name].double() - want).norm() / want.norm())
        assert rel < most, f"{name}: {rel:.2e} of {most:.2e}"


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,hidden,inner", [(1, 256, 704), (37, 256, 704), (300, 512, 1408), (700, 333, 1001)])
def test_gradients(tokens, hidden, inner, dtype, layer):
    w, x, r, d = block(tokens, hidden, inner, dtype, layer)
    _, kept = mlp_train.forward(x, r, w)
    got = mlp_train.backward(d, kept, w)
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0
    check(got, mlp_train.gradients64(d, x, r, w), dtype)


@pytest.mark.parametrize("layer", [False, True])
def test_in_a_graph(layer):
    """One step captured; replayed with other inputs, it gives what the calls give."""
    w, x, r, d = block(130, 256, 704, torch.bfloat16, layer)
    mlp_train.backward(d, mlp_train.forward(x, r, w)[1], w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, kept = mlp_train.forward(x, r, w)
        got = mlp_train.backward(d, kept, w)
    for seed in (7, 8):
        for t, s in ((x, seed), (r, seed + 10), (d, seed + 20)):
            t.copy_(rand(t.shape, s, t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        out2, kept2 = mlp_train.forward(x, r, w)
        want = mlp_train.backward(d, kept2, w)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and all(torch.equal(got[k], want[k]) for k in want)


def test_two_graphs_and_an_eager_step():
    """Two captured steps with memory of their own and eager calls between do not disturb each other."""
    a, b = block(64, 256, 704, torch.float16, False, 1), block(200, 320, 512, torch.float16, True, 5)
    want = [mlp_train.backward(d, mlp_train.forward(x, r, w)[1], w) for w, x, r, d in (a, b)]
    graphs, got = [], []
    for w, x, r, d in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(mlp_train.backward(d, mlp_train.forward(x, r, w)[1], w))
    for _ in range(3):
        graphs[0].replay()
        w, x, r, d = b
        eager = mlp_train.backward(d, mlp_train.forward(x, r, w)[1], w)
        graphs[1].replay()
    torch.cuda.synchronize()
    for g, t in ((got[0], want[0]), (got[1], want[1]), (eager, want[1])):
        assert all(torch.equal(g[k], t[k]) for k in t)


CALLS = {
    "layernorm": lambda t, **k: bg.layernorm(t["x"], t["v"], t["v"], residual=t["x2"], **k),
    "layernorm to mx": lambda t, **k: bg.layernorm(t["x"], out_dtype=torch.float8_e4m3fn, **k),
    "layernorm_backward": lambda t, **k: bg.layernorm_backward(t["x2"], t["x"], t["m"], t["m"], t["v"], **k),
    "rmsnorm_backward": lambda t, **k: bg.rmsnorm_backward(t["x2"], t["x"], t["v"], **k),
    "matmul_gated": lambda t, **k: bg.matmul_gated(t["x"], t["w"], t["w2"], **k),
    "matmul_backward": lambda t, **k: bg.matmul_backward(t["d"], t["x"], t["w"], **k),
    "matmul_gated_backward": lambda t, **k: bg.matmul_gated_backward(t["d"], t["x"], t["w"], t["w2"], t["g"], t["u"], **k),
}


def operands():
    M, N, K = 70, 390, 1025              # rows off the 16-byte grid
    t = {"x": rand((M, K), 1, torch.bfloat16), "x2": rand((M, K), 2, torch.bfloat16), "w": rand((N, K), 3, torch.bfloat16),
         "w2": rand((N, K), 4, torch.bfloat16), "d": rand((M, N), 5, torch.bfloat16), "g": rand((M, N), 6, torch.bfloat16),
         "u": rand((M, N), 7, torch.bfloat16), "v": rand((K,), 8, torch.float32), "m": rand((M,), 9, torch.float32)}
    return t


def same(a, b):
    a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
    return all(torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_on_another_stream_while_the_current_one_is_busy(name, handle):
    t = operands()
    want = CALLS[name](t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    filled = [torch.empty(n, dtype=torch.uint8, device="cuda")
              for n in (4 << 10, 64 << 10, 100 << 10, 200 << 10, 600 << 10, 1 << 20, 2 << 20, 4 << 20) for _ in range(3)]
    torch.cuda._sleep(40_000_000)         # cycles: about 20 ms
    for f in filled:
        f.fill_(255)
    del filled, f
    got = [CALLS[name](t, stream=s.cuda_stream if handle else s) for _ in range(4)]
    s.synchronize()
    early = [tuple(v.clone() for v in (g if isinstance(g, tuple) else (g,))) for g in got]     # behind the pending writes
    torch.cuda.synchronize()
    for g, e in zip(got, early):
        assert same(g, want) and same(e, want)
    assert bg.bigemm_last_device_error() == 0


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_two_streams_at_once(name):
    """Each call has its own workspace: calls in flight together give what they give alone."""
    t = operands()
    want = CALLS[name](t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(CALLS[name](t))
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)
