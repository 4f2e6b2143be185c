"""Layer calls of several threads at once, each on a stream of its own: the results of calls one after the other."""
import threading

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu


def rand(shape, seed, kind):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(kind)


def work(seed):
    """Calls of every kernel of the training operators, and what they give."""
    kind = torch.float16 if seed % 2 else torch.bfloat16
    out = []
    for M, N, K in ((4, 300, 264), (300, 712, 520), (100, 77, 201)):
        x, wg, wu, d = (rand(s, seed + i, kind) for i, s in enumerate(((M, K), (N, K), (N, K), (M, N))))
        g, u = torch.empty_like(d), torch.empty_like(d)
        db, dg, du = (torch.empty(N, device="cuda") for _ in range(3))
        out += [bg.matmul(x, wg), bg.matmul_gated(x, wg, wu, gate_out=g, up_out=u), g, u]
        out += [*bg.matmul_gated_backward(d, x, wg, wu, g, u, dbias_gate=dg, dbias_up=du), dg, du]
        out += [*bg.matmul_backward(d, x, wg, dbias=db), db]
    for rows, cols in ((40, 200), (60, 1001), (30, 9000), (20, 20001)):
        x, d = rand((rows, cols), seed, kind), rand((rows, cols), seed + 1, kind)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        out += [bg.layernorm(x, mean_out=mean, rstd_out=rstd), *bg.layernorm_backward(d, x, mean, rstd), *bg.rmsnorm_backward(d, x)]
    return out


def test_threads():
    count = 6
    want = [work(s) for s in range(count)]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(count)

    def run(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for turn in range(8):
                    for i, (a, b) in enumerate(zip(want[seed], work(seed))):
                        if not torch.equal(a, b):
                            wrong.append((seed, turn, i))
        except Exception as e:
            wrong.append((seed, repr(e)))

    threads = [threading.Thread(target=run, args=(s,)) for s in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and bg.bigemm_last_device_error() == 0
