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
    return torch.full(shape, 0, dtype=dtype).as_subclass(Cuda)  # (not one of the recorded functions)


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
                if name == "w12_kv4_page_bytes":
                    return args[0] * args[2] * (args[1] + 8)
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
    w12.logprobs(cuda(4, 100), k=3, stream=Stream())
    assert len(made) == 6 and all(on for _, on in made), made
    assert launched == [("w12_logprobs", 5)]


def _weights(N, K):
    u8 = dict(dtype=torch.uint8)
    return w12.W12Weights(N, K, *(cuda(N, K // 2, **u8) for _ in range(3)), cuda(K // 128, N, **u8),
                          cuda((N // 128) * (K // 128) + 1, dtype=torch.int32), cuda(1, dtype=torch.int32), 0)


def _i32(*shape):
    return cuda(*shape, dtype=torch.int32)


def _bf16(*shape):
    return cuda(*shape, dtype=torch.bfloat16)


CALLS = {
    "pack": lambda s: w12.pack(_bf16(256, 128), stream=s),
    "unpack": lambda s: w12.unpack(_weights(256, 128), stream=s),
    "gemm": lambda s: w12.gemm(_bf16(4, 128), _weights(256, 128), stream=s),
    "gemm_bf16_ref": lambda s: w12.gemm_bf16_ref(_bf16(4, 128), _bf16(256, 128), stream=s),
    "verify_greedy": lambda s: w12.verify_greedy(cuda(4, 256), _i32(1, 4), 4, stream=s),
    "verify_greedy_fused": lambda s: w12.verify_greedy_fused(_bf16(4, 128), _weights(256, 128), _i32(1, 4), 4, stream=s),
    "verify_tree": lambda s: w12.verify_tree(cuda(4, 256), _i32(1, 4), _i32(1, 4), stream=s),
    "verify_tree_fused": lambda s: w12.verify_tree_fused(_bf16(4, 128), _weights(256, 128), _i32(1, 4), _i32(1, 4), stream=s),
    "kv_commit": lambda s: w12.kv_commit([_bf16(2, 8, 16)], _i32(2), _i32(2, 4), _i32(2), stream=s),
    "state_select": lambda s: w12.state_select(_bf16(2, 4, 16), _i32(2, 4), _i32(2), stream=s),
    "tree_attention": lambda s: w12.tree_attention(_bf16(2, 4, 2, 128), _bf16(2, 8, 1, 128), _bf16(2, 8, 1, 128), _i32(2),
                                                   _i32(2, 4), stream=s),
    "kv4_commit": lambda s: w12.kv4_commit([w12.KV4Cache(cuda(1, 1, 16 * 72, dtype=torch.uint8), 16, 64)], _i32(2, 1), _i32(2),
                                           _i32(2, 4), _i32(2), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_every_function_that_takes_a_stream(record, name):
    made, launched = record
    CALLS[name](Stream())
    assert made and all(on for _, on in made), made
    assert launched and all(stream == 5 for _, stream in launched)
