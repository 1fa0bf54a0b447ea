"""Waits of the serving operators that expire: the call ends, says so, and leaves nothing
behind that another kernel could meet."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")

DEFAULT_US = 2000000


@pytest.fixture
def short_waits():
    torch.cuda.synchronize()
    w12.set_wait_limit_us(1)
    yield
    torch.cuda.synchronize()
    w12.set_wait_limit_us(DEFAULT_US)


@pytest.mark.parametrize("T,prefix", [(1, [60, 200, 500]), (3, [300] * 40), (16, [60, 200, 350]), (40, [130] * 40)])
def test_runs_of_no_more_blocks_than_stages(short_waits, T, prefix):
    """Every copy of a run is issued at once, so waits for them may expire after the
    copying warp is through. Kernels that use the same shared memory next are right."""
    B = len(prefix)
    c = Case(prefix, [T] * B, T, 10, 2, 128, 64, seed=T)
    att = w12.KV4Attention(B, T, 10, 2, 128, 64, max(prefix) + T)
    args = (c.Q, c.cache, to_dev_i32(c.table), to_dev_i32(c.prefix))
    V = 20000
    x = torch.randn((8, V), device="cuda")
    want = torch.log_softmax(x.double(), 1)
    lp = w12.TokenLogprobs(8, V, 4)
    tokens = to_dev_i32(np.arange(8)[:, None])
    torch.cuda.synchronize()
    for _ in range(8):
        st = new_status()
        w12.set_wait_limit_us(1)
        att.run(*args, status=st)
        w12.set_wait_limit_us(DEFAULT_US)              # (for the launches from here on)
        st2 = new_status()
        got = lp.run(x, tokens, status=st2)[0]
        assert status_value(st2) == 0
        assert (got[:, 0].double() - want[torch.arange(8), torch.arange(8)]).abs().max() < 1e-4
        code = status_value(st)
        assert code in (0, 6)
        if code:
            att.reset()
    st = new_status()
    c.check(att.run(*args, status=st))
    assert status_value(st) == 0


# Runs of many blocks: with a bound of 1 us some wait expires in every call (10 are given).
LONG = [(3, [8000] * 40, 16, 8, 128), (16, [9000] * 8, 8, 8, 128), (40, [9000] * 8, 10, 2, 128), (40, [9000] * 8, 10, 2, 64)]


def until_expired(call, reset):
    for _ in range(10):
        st = new_status()
        torch.cuda.synchronize()
        w12.set_wait_limit_us(1)
        call(st)
        w12.set_wait_limit_us(DEFAULT_US)
        code = status_value(st)
        reset()
        assert code in (0, 6)
        if code == 6:
            return
    raise AssertionError("no wait expired")


@pytest.mark.parametrize("T,prefix,Hq,Hkv,d", LONG)
def test_attention_over_long_caches(short_waits, T, prefix, Hq, Hkv, d):
    B = len(prefix)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = prefix[0] + T
    width = -(-n // 64)
    cache = w12.KV4Cache.create(B * width, Hkv, d, 64)
    pages = w12.PageTable.create(B, width, B * width, 64)
    length = torch.full((B,), n, dtype=torch.int32, device="cuda")
    slots = pages.reserve(torch.zeros_like(length), length, n).flatten()
    K, V = (torch.randn((B * n, Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache.append(K, V, slots)
    Q = torch.randn((B, T, Hq, d), generator=g, device="cuda").bfloat16()
    att = w12.KV4Attention(B, T, Hq, Hkv, d, 64, n)
    args = Q, cache, pages.table, length - T
    w12.set_wait_limit_us(DEFAULT_US)
    want = att.run(*args)
    torch.cuda.synchronize()
    for _ in range(3):
        until_expired(lambda st: att.run(*args, status=st), att.reset)
        st = new_status()
        assert torch.equal(att.run(*args, status=st), want) and status_value(st) == 0


@pytest.mark.parametrize("M,V,k,dtype", [(600, 151936, 0, torch.bfloat16), (256, 151936, 8, torch.float32)])
def test_log_probabilities_of_many_rows(short_waits, M, V, k, dtype):
    a = w12.TokenLogprobs(M, V, k)
    x = torch.randn((M, V), device="cuda").to(dtype)
    tokens = to_dev_i32(np.arange(M)[:, None])
    w12.set_wait_limit_us(DEFAULT_US)
    want = a.run(x, tokens)
    torch.cuda.synchronize()
    for _ in range(3):
        until_expired(lambda st: a.run(x, tokens, status=st), a.ws.zero_)
        st = new_status()
        assert all(torch.equal(p, q) for p, q in zip(a.run(x, tokens, status=st), want)) and status_value(st) == 0
