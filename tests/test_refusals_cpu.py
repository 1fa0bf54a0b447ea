"""Arguments that the binding refuses before anything reaches the library, on the CPU: the
library is replaced by one that accepts everything, CPU tensors pass for CUDA ones."""
import pytest
import torch

from speculative_decoding_verification_w12_gb300 import w12
from test_streams_cpu import cuda


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Lib:
        def w12_kv4_page_bytes(self, Hkv, d, P):
            return Hkv * P * (d + 8)

        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0

    monkeypatch.setattr(w12, "lib", lambda: Lib())
    monkeypatch.setattr(w12, "_stream", lambda stream=None: 0)
    return made


def i32(*shape):
    return cuda(*shape, dtype=torch.int32)


def test_commit_refuses_lengths_that_it_would_write_past(calls):
    cache = w12.KV4Cache(cuda(2, 1, 16 * 72, dtype=torch.uint8), 16, 64)
    args = [cache], i32(3, 2), i32(3), i32(3, 4), i32(3)
    good = i32(3)
    assert w12.kv4_commit(*args, new_len=good) is good and calls == ["w12_kv4_commit"]
    for bad in (i32(2), i32(3, 1), cuda(3, dtype=torch.int64), i32(6)[::2], torch.full((3,), 0, dtype=torch.int32), args[2]):
        with pytest.raises(ValueError):
            w12.kv4_commit(*args, new_len=bad)
    assert calls == ["w12_kv4_commit"]
