"""Memory that a call makes for itself belongs to the stream that the call runs on: made
on another, the allocator may hand it out again while the kernel is running, and a zero
fill of it is not ordered before the kernel. Checked on the CPU, with the library and the
stream context replaced by recorders."""
import pytest
import torch

from speculative_decoding_verification_w12_gb300 import w12


class Cuda(torch.Tensor):
    """A CPU tensor that passes for a CUDA one."""
    is_cuda = property(lambda self: True)


def cuda(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)


class Stream:
    cuda_stream = 5


@pytest.fixture
def record(monkeypatch):
    """Allocations of a call: (what, whether within the context of the call's stream)."""
    inside, made, launched = [], [], []

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *exc):
            inside.pop()

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_ws_bytes"):
                    return 512
                launched.append((name, args[-1]))
                return 0
            return call

    def recorded(name):
        real = getattr(torch, name)

        def make(*args, **kw):
            made.append((name, bool(inside) and isinstance(inside[-1], Stream)))
            return real(*args, **kw)
        return make

    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(w12, "lib", lambda: Lib())
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(name))
    return made, launched


def test_log_probabilities(record):
    made, launched = record
    x = cuda(4, 100)
    made.clear()
    w12.logprobs(x, k=3, stream=Stream())
    assert len(made) == 6 and all(on for _, on in made), made
    assert launched == [("w12_logprobs", 5)]
