"""Calls on a stream that is not the current one, with the current stream busy allocating
and filling memory of the sizes that the calls make for themselves."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")


def beside(call, sizes, times=12):
    """call(stream) several times on a side stream; after each, blocks of the given sizes are
    allocated on the current stream and filled. Returns the results."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = []
    for _ in range(times):
        out.append(call(side))
        junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        del junk
    side.synchronize()
    torch.cuda.synchronize()
    return out


def test_log_probabilities_in_one_call():
    M, V, k = 64, 60000, 8
    x = torch.randn((M, V), device="cuda")
    tokens = to_dev_i32(np.arange(M)[:, None])
    want = w12.TokenLogprobs(M, V, k).run(x, tokens)
    st = new_status()
    size = w12.TokenLogprobs(M, V, k).ws.numel()
    for got in beside(lambda s: w12.logprobs(x, tokens, k, status=st, stream=s), [size, M * k * 4, M * 4]):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert status_value(st) == 0
