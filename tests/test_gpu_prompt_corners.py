"""Prompt attention where a call's form must not show: values that are not finite beside weights that
vanish, and waits that expire."""
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from speculative_decoding_verification_w12_gb300 import w12
from test_gpu_expired_waits import short_waits, until_expired  # noqa: F401
from test_gpu_prompt_attention import BF16, F16, _offsets, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("G,d", [(1, 64), (1, 128), (2, 64), (4, 128), (5, 64), (8, 128)])
def test_values_beside_weights_that_vanish(G, d, dtype):
    """Every tenth key has a value that is not finite and scores so low that its weight is zero in fp32: at every
    place in a tile, so also where only the first of an item's two tiles is cut by the diagonal. Many kv heads
    make items of two tiles, each by itself items of one: the same bits."""
    lens, Hkv = [700, 0, 333, 16, 129], 16
    cu = _offsets(lens)
    q, k, v = _rows(sum(lens), Hkv * G, Hkv, d, dtype, G + d)
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    k[3::10, :, 0] = -4000.0                                 # scores of -32,000 times the scale: 2^-4000 and less
    for i, bad in enumerate((float("inf"), float("nan"), float("-inf"))):
        v[3 + 10 * i::30, :, 5 + i] = bad
    dev, st = to_dev_i32(cu), new_status()
    out = w12.prompt_attention(q, k, v, dev, status=st)
    assert status_value(st) == 0
    for h in range(Hkv):
        heads = slice(h * G, h * G + G)
        one = w12.prompt_attention(q[:, heads], k[:, h:h + 1], v[:, h:h + 1], dev)
        same = (out[:, heads] == one) | (torch.isnan(out[:, heads]) & torch.isnan(one))
        assert same.all(), (h, torch.nonzero(~same)[0].tolist())
    # A row that sees such a value is not finite there, and in no other column.
    start = torch.cat([torch.full((n,), a) for a, n in zip(cu, lens)]).cuda()
    rows = torch.arange(sum(lens), device="cuda")
    for i in range(3):
        at = torch.arange(3 + 10 * i, sum(lens), 30, device="cuda")
        sees = ((at[None] >= start[:, None]) & (at[None] <= rows[:, None])).any(1)
        assert torch.equal(torch.isfinite(out[..., 5 + i]).all(1), ~sees) and torch.equal(torch.isfinite(out[..., 5 + i]).any(1), ~sees)
    assert torch.isfinite(out[..., 8:]).all()


@pytest.mark.parametrize("lens,Hq,Hkv,d,dtype", [([1900, 2000], 40, 8, 128, BF16), ([6000], 32, 8, 64, F16), ([500] * 40, 16, 8, 64, BF16)])
def test_a_bound_of_a_microsecond_expires(short_waits, lens, Hq, Hkv, d, dtype):  # noqa: F811
    q, k, v = _rows(sum(lens), Hq, Hkv, d, dtype, 6)
    cu = to_dev_i32(_offsets(lens))
    w12.set_wait_limit_us(2000000)
    want = w12.prompt_attention(q, k, v, cu)
    torch.cuda.synchronize()
    for _ in range(3):
        until_expired(lambda st: w12.prompt_attention(q, k, v, cu, status=st), lambda: None)
        st = new_status()
        assert torch.equal(w12.prompt_attention(q, k, v, cu, status=st), want) and status_value(st) == 0
