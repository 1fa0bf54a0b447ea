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
