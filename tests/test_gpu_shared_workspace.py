"""One workspace under calls of different sizes and operators: the paged attention and the
log probabilities leave nothing in it that another of their calls could mistake."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")


class Logprobs:
    def __init__(self, M, V, k, dtype=torch.float32):
        g = torch.Generator(device="cuda").manual_seed(M + V)
        self.x = (torch.randn((M, V), generator=g, device="cuda") * 3).to(dtype)
        self.tokens = to_dev_i32(np.arange(M)[:, None] % V)
        self.op = w12.TokenLogprobs(M, V, k)
        self.want = [t.clone() for t in self.run()]

    def run(self):
        st = new_status()
        out = self.op.run(self.x, self.tokens, status=st)
        assert status_value(st) == 0
        return out


class Attention:
    def __init__(self, prefix, T, Hq, Hkv, d, tree=False):
        self.c = Case(prefix, [T] * len(prefix), T, Hq, Hkv, d, 64, seed=T + d)
        if tree:
            self.c.trees()
        self.op = w12.KV4Attention(len(prefix), T, Hq, Hkv, d, 64, max(prefix) + T)
        self.want = [self.run()[0].clone()]
        self.c.check(self.want[0])

    def run(self):
        st = new_status()
        out = self.c.run(att=self.op, status=st, out=torch.full_like(self.c.Q, float("nan")))
        assert status_value(st) == 0
        return [out]


def test_calls_of_any_size_and_both_operators_take_turns():
    ops = [Logprobs(16, 151936, 20), Logprobs(256, 30000, 8, torch.bfloat16), Logprobs(1, 100, 0), Logprobs(700, 9000, 32),
           Attention([3000, 50], 1, 10, 2, 128), Attention([777], 1, 40, 8, 128), Attention([900] * 60, 1, 8, 8, 64),
           Attention([2000, 70], 40, 10, 2, 128, tree=True), Attention([300] * 30, 33, 8, 4, 64)]
    ws = w12.workspace(max(o.op.ws.numel() for o in ops))
    for o in ops:
        o.op.ws = ws
    order = np.random.default_rng(0)
    for i in [*range(len(ops)), *reversed(range(len(ops))), *order.integers(0, len(ops), 40)]:
        for got, want in zip(ops[i].run(), ops[i].want):
            assert torch.equal(got, want), i


def test_rows_of_one_call_on_a_used_workspace():
    """A small call, then a large one whose counters once lay where the small one's partial
    results do."""
    small, large = Logprobs(16, 60000, 0), Logprobs(256, 60000, 0)
    small.op.ws = large.op.ws
    small.run()
    for got, want in zip(large.run(), large.want):
        assert torch.equal(got, want)
