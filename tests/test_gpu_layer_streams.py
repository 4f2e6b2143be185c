"""Layer calls on a stream of their own while the current one is busy: outputs, scales and workspaces that a call makes
neither wait for the current stream's pending work nor meet it in memory."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

MX = torch.float8_e4m3fn


def rand(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def operands():
    x, w = rand((70, 1025), 1, torch.bfloat16), rand((390, 1025), 2, torch.bfloat16)     # rows off the 16-byte grid
    q, s = bg.mx_quantize(rand((70, 1040), 3, torch.float32))
    p, t = bg.mx_quantize(rand((390, 1040), 4, torch.float32))
    return x, w, (q, s), (p, t)


CALLS = {
    "matmul": lambda o, **k: bg.matmul(o[0], o[1], **k),
    "matmul_mx": lambda o, **k: bg.matmul_mx(*o[2], *o[3], **k),
    "matmul_mx to mx": lambda o, **k: bg.matmul_mx(*o[2], *o[3], out_dtype=MX, **k),
    "rmsnorm": lambda o, **k: bg.rmsnorm(o[0], residual=o[0], **k),
    "rmsnorm to mx": lambda o, **k: bg.rmsnorm(o[0], out_dtype=MX, **k),
    "mx_quantize": lambda o, **k: bg.mx_quantize(o[0], **k),
}


def tensors(got):
    return [t for t in (got if isinstance(got, tuple) else (got,))]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(tensors(a), tensors(b)))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_while_the_current_stream_is_busy(name, handle):
    o = operands()
    want = CALLS[name](o)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    # blocks of every size that the call may ask for, freed here with writes to them still pending
    filled = [torch.empty(n, dtype=torch.uint8, device="cuda")
              for n in (64 << 10, 100 << 10, 200 << 10, 600 << 10, 800 << 10, 1 << 20, 2 << 20) for _ in range(3)]
    torch.cuda._sleep(40_000_000)         # cycles: about 20 ms
    for f in filled:
        f.fill_(255)
    del filled, f
    got = [CALLS[name](o, stream=s.cuda_stream if handle else s) for _ in range(4)]
    s.synchronize()
    early = [[t.clone() for t in tensors(g)] for g in got]     # behind the pending writes
    torch.cuda.synchronize()
    for g, e in zip(got, early):
        assert same(g, want) and same(tuple(e), want)
    assert bg.bigemm_last_device_error() == 0


def test_returned_tensors_outlive_their_use():
    """A result freed while the current stream still reads it is not given to the next call on the other stream."""
    o = operands()
    want, other = bg.matmul(o[0], o[1]), -o[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = bg.matmul(o[0], o[1], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(40_000_000)
    kept = y.clone()
    del y
    for _ in range(4):
        bg.matmul(other, o[1], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
