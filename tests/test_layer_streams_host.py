"""What a layer call with `stream=` allocates is made on that stream, without a GPU: torch's streams and the extension
module are fakes that keep a record, and tensors lie on the CPU."""
import contextlib

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

MX = torch.float8_e4m3fn


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Record:
    """made: (what, the stream that was current); recorded: streams of record_stream calls; given: of the calls."""

    def __init__(self):
        self.current, self.made, self.recorded, self.given = "caller", [], [], []


class FakeModule:
    def __init__(self, rec):
        self.rec = rec

    def product(self, x, x_scale, w, w_scale, bias, act, other, combine, out, out_scale, stream):
        bg._workspace(4096, x, stream)       # as for operands off the 16-byte grid
        self.rec.given.append(stream)
        return 0

    def norm(self, *args):
        self.rec.given.append(args[-1])
        return 0

    quantize = norm


@pytest.fixture
def rec(monkeypatch):
    r = Record()

    @contextlib.contextmanager
    def on(stream):
        before, r.current = r.current, stream
        yield
        r.current = before

    def making(make):
        def call(*args, **kw):
            r.made.append((make.__name__, r.current))
            return make(*args, **kw)
        call.__name__ = make.__name__
        return call

    monkeypatch.setattr(bg, "_layer_module", FakeModule(r))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: r.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: r.recorded.append(s))
    monkeypatch.setattr(torch, "empty", making(torch.empty))
    monkeypatch.setattr(torch, "zeros", making(torch.zeros))
    return r


X, W = torch.ones(3, 33, dtype=torch.float16), torch.ones(5, 33, dtype=torch.float16)
Q, P = torch.ones(3, 32).to(MX), torch.ones(5, 32).to(MX)
S = torch.ones(512, dtype=torch.uint8)
# the call, and how many tensors it makes and returns
CALLS = {
    "matmul": (lambda **k: bg.matmul(X, W, **k), 2, 1),
    "matmul_mx": (lambda **k: bg.matmul_mx(Q, S, P, S, **k), 2, 1),
    "matmul_mx to mx": (lambda **k: bg.matmul_mx(Q, S, P, S, out_dtype=MX, **k), 3, 2),
    "rmsnorm": (lambda **k: bg.rmsnorm(X, **k), 1, 1),
    "rmsnorm to mx, residual": (lambda **k: bg.rmsnorm(X, residual=X, out_dtype=MX, **k), 3, 3),
    "mx_quantize": (lambda **k: bg.mx_quantize(X, **k), 2, 2),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", ["stream", "address", "default", "object"])
def test_made_on_the_calls_stream(rec, name, given):
    call, made, returned = CALLS[name]
    stream = {"stream": FakeStream(4096), "address": 8192, "default": 0,
              "object": type("Other", (), {"cuda_stream": 8192})()}[given]
    on = {"stream": stream, "address": ("external", 8192), "default": "default", "object": ("external", 8192)}[given]
    call(stream=stream)
    assert len(rec.made) == made and all(s is on or s == on for _, s in rec.made), rec.made
    assert rec.recorded == ["caller"] * returned         # what is returned is used on the caller's stream
    assert rec.given == [stream]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream(rec, name):
    call, made, _ = CALLS[name]
    call()
    assert [s for _, s in rec.made] == ["caller"] * made and rec.recorded == [] and rec.given == [None]
