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


def test_gemm_and_tree_attention_in_one_call():
    g = torch.Generator(device="cuda").manual_seed(0)
    W = w12.pack(torch.randn((1024, 512), generator=g, device="cuda").bfloat16())
    X = torch.randn((16, 512), generator=g, device="cuda").bfloat16()
    ws = w12.workspace(w12.gemm_ws_bytes(16, 1024, 512))
    want = w12.gemm(X, W, ws=ws)
    for got in beside(lambda s: w12.gemm(X, W, stream=s), [ws.numel(), want.numel() * 4]):
        assert torch.equal(got, want)
    B, T, Hq, Hkv, S = 2, 16, 10, 2, 600
    Q, K, V = (torch.randn(shape, generator=g, device="cuda").bfloat16()
               for shape in ((B, T, Hq, 128), (B, S, Hkv, 128), (B, S, Hkv, 128)))
    prefix, parents = to_dev_i32([500, 37]), to_dev_i32([list(range(-1, T - 1))] * B)
    att = w12.TreeAttention(B, T, Hq, Hkv, S)
    want = att.run(Q, K, V, prefix, parents)
    for got in beside(lambda s: w12.tree_attention(Q, K, V, prefix, parents, stream=s), [att.ws.numel(), want.numel() * 2]):
        assert torch.equal(got, want)
