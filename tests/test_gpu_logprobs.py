"""GPU log probabilities, entropy and top alternatives against the float64 oracle.

Tolerances: x = scale * logit is one fp32 rounding that the oracle makes too.
lse: the sum of V positive fp32 terms in chunks of at most 64 per thread, then
trees: a relative error of (64 + 32 + a few) 2^-24 plus 2^-22 for each
exponential, so under 2^-16 in the sum and 2^-16 absolute in its logarithm, plus
a rounding of lse itself. A logprob adds one subtraction (2^-24 of lse).
entropy = log S0 - S1 / S0: S1's terms have one sign, so its relative error is
as S0's: 2^-16 of the (positive) mean of -t, plus that of log S0.
"""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")

TOL = 2.0 ** -16


def _check(x, scale, tokens, k, out):
    lp, ent, lse, top, ids = (t.cpu().numpy() for t in out)
    rlp, rent, rlse, rtop, rids = O.logprobs(x.float().cpu().numpy(), scale, tokens, k)
    big = np.abs(np.where(np.isfinite(rlse), rlse, 0)) + 1          # of each row
    mag = np.abs(np.where(np.isfinite(rlp), rlp, 0))
    tol = TOL + 2.0 ** -22 * big
    assert (np.isinf(lse) == np.isinf(rlse)).all()
    assert (np.abs(np.where(np.isinf(rlse), 0, lse) - np.where(np.isinf(rlse), 0, rlse)) <= tol).all()
    assert (np.isinf(lp) == np.isinf(rlp)).all()
    assert (np.abs(np.where(np.isinf(rlp), 0, lp - np.where(np.isinf(rlp), 0, rlp))) <= tol[:, None] + 2.0 ** -22 * mag).all()
    # The mean of -t is entropy - (lse - max) <= entropy.
    assert (np.abs(ent - rent) <= tol + TOL * rent).all()
    assert (ids == rids).all()
    fin = np.isfinite(rtop)
    assert (np.isfinite(top) == fin).all() and (top[~fin] == -np.inf).all()
    off = np.abs(np.where(fin, top, 0) - np.where(fin, rtop, 0))
    assert (off <= tol[:, None] + 2.0 ** -22 * np.abs(np.where(fin, rtop, 0))).all()


def _run(x, tokens, k, scale=1.0):
    st = new_status()
    out = w12.logprobs(x, to_dev_i32(tokens), k, scale, status=st)
    assert status_value(st) == 0
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,V,n,k,scale", [(1, 1, 1, 1, 1.0), (3, 7, 2, 32, 0.7), (16, 4096, 1, 20, 1.0), (5, 4097, 3, 5, 1.25),
                                           (2, 16385, 1, 1, 3.0), (1, 151936, 4, 32, 1.0), (70, 151936, 1, 20, 0.5), (33, 32001, 2, 8, 1.0)])
def test_rows_match_the_oracle(M, V, n, k, scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + V)
    x = (torch.randn((M, V), generator=g, device="cuda") * 3).to(dtype)
    tokens = np.random.default_rng(V).integers(0, V, (M, n))
    if n > 1:
        tokens[0, 1] = -1
    _check(x, scale, tokens, k, _run(x, tokens, k, scale))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_with_padded_and_unaligned_rows(dtype):
    x = torch.randn((6, 5003), device="cuda").to(dtype)
    for off, width in ((0, 5000), (1, 4999), (3, 4000), (8, 4096)):
        v = x[:, off:off + width]
        tokens = np.arange(6)[:, None] * 3
        _check(v, 1.0, tokens, 10, _run(v, tokens, 10))


def test_masked_tokens_and_empty_rows():
    x = torch.randn((8, 40000), device="cuda")
    x[0] = -np.inf
    x[1, 5:] = -np.inf                                   # five tokens left of a list of ten
    x[2, :39999] = -np.inf                               # one
    x[3] = torch.finfo(torch.float32).min                # the lowest value everywhere: uniform
    x[4, 100:] = torch.finfo(torch.float32).min          # in masked places
    x[5, ::2] = -np.inf
    x[6, :20000] = -np.inf
    tokens = np.array([[0, 1], [0, 9], [39999, 3], [7, 8], [5, 39999], [1, 2], [20000, 0], [1, -1]])
    _check(x, 1.0, tokens, 10, _run(x, tokens, 10))
    _check(x[4:], 2.5, tokens[4:], 10, tuple(t[4:] for t in _run(x, tokens, 10, 2.5)))   # lowest * 2.5 is -inf


@pytest.mark.parametrize("V", [300, 20000, 151936])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two", "zeros", "few"])
def test_ties_and_orders_that_flood_the_candidates(kind, V):
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"equal": torch.full((V,), 2.0, device="cuda"), "rising": i / V, "falling": -i / V, "two": (i % 2),
           "zeros": torch.where(i % 2 == 0, 0.0, -0.0), "few": torch.where(i % 977 < 40, i / V, torch.full_like(i, -np.inf))}[kind]
    x = torch.stack([row, row.flip(0)])
    tokens = np.array([[0], [V - 1]])
    for k in (1, 20, 32):
        _check(x, 1.0, tokens, k, _run(x, tokens, k))


def test_nan_and_inf_rows():
    x = torch.randn((4, 9000), device="cuda")
    x[0, 17] = np.nan
    x[1, 8999] = np.inf
    tokens = np.array([[3], [3], [3], [3]])
    lp, ent, lse, top, ids = _run(x, tokens, 4)
    assert torch.isnan(lp[0]).all() and torch.isnan(ent[0]) and torch.isnan(lse[0]) and torch.isnan(top[0]).all()
    assert torch.isnan(lse[1]) and torch.isnan(ent[1]) and ids[1, 0] == 8999
    _check(x[2:], 1.0, tokens[2:], 4, (lp[2:], ent[2:], lse[2:], top[2:], ids[2:]))


def test_large_logits_do_not_overflow():
    x = torch.randn((2, 5000), device="cuda") * 1e4
    x[1] += 1e30
    tokens = np.array([[1], [2]])
    lp, ent, lse, top, ids = _run(x[:1].contiguous(), tokens[:1], 3)
    assert torch.isfinite(lse).all() and float(top[0, 0]) == 0.0 and float(ent[0]) == 0.0
    assert int(ids[0, 0]) == int(x[0].argmax())
    out = _run(x[1:].contiguous(), tokens[1:], 3)
    assert abs(float(out[1][0]) - np.log(5000)) < 1e-4     # 1e30 swallows the rest: a uniform row


def test_no_tokens_no_list():
    x = torch.randn((3, 1000), device="cuda")
    lp, ent, lse, top, ids = w12.logprobs(x)
    assert lp.shape == (3, 0) and top.shape == (3, 0) and ids.shape == (3, 0)
    _check(x, 1.0, np.zeros((3, 0), dtype=int), 0, (lp, ent, lse, top, ids))


def test_bad_tokens_are_flagged():
    x = torch.randn((2, 1000), device="cuda")
    st = new_status()
    lp = w12.logprobs(x, to_dev_i32([[1000, 5], [-2, -1]]), status=st)[0]
    assert status_value(st) == 1
    assert torch.isnan(lp[0, 0]) and torch.isnan(lp[1, 0]) and torch.isfinite(lp[0, 1]) and lp[1, 1] == 0


def test_workspace_reused_streams_and_graph():
    a = w12.TokenLogprobs(9, 50000, 12)
    tokens = to_dev_i32(np.arange(18).reshape(9, 2))
    x = torch.randn((9, 50000), device="cuda")
    first = [t.clone() for t in a.run(x, tokens)]
    for _ in range(3):
        assert all((p == q).all() for p, q in zip(a.run(x, tokens), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = a.run(x, tokens, stream=s)
    s.synchronize()
    assert all((p == q).all() for p, q in zip(out, first))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = a.run(x, tokens)
    x.copy_(torch.randn_like(x))
    g.replay()
    torch.cuda.synchronize()
    _check(x, 1.0, tokens.cpu().numpy(), 12, out)


def test_binding_refusals():
    a = w12.TokenLogprobs(4, 100, 3)
    x = torch.zeros((4, 100), device="cuda")
    with pytest.raises(TypeError):
        a.run(x.double())
    for bad in (x[:3], x.t().contiguous().t(), x.cpu()):
        with pytest.raises(ValueError):
            a.run(bad)
    with pytest.raises(ValueError):
        a.run(x, torch.zeros((4, 1), dtype=torch.int64, device="cuda"))
    with pytest.raises(w12.W12Error) as e:
        a.run(x, scale=-1.0)
    assert e.value.code == 1
    with pytest.raises(w12.W12Error) as e:
        w12.TokenLogprobs(4, 100, 33)
    assert e.value.code == 2


def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    a = w12.TokenLogprobs(40, 60000, 5)
    x = torch.randn((40, 60000), device="cuda")
    tokens = np.arange(40)[:, None]
    torch.cuda.synchronize()
    w12.set_wait_limit_us(1)
    try:
        st = new_status()
        out = a.run(x, to_dev_i32(tokens), status=st)
        code = status_value(st)
    finally:
        w12.set_wait_limit_us(2000000)
    assert code in (0, 6)
    if code == 0:
        _check(x, 1.0, tokens, 5, out)
    a.ws.zero_()
    st = new_status()
    out = a.run(x, to_dev_i32(tokens), status=st)
    assert status_value(st) == 0
    _check(x, 1.0, tokens, 5, out)


@pytest.mark.parametrize("kind", ["rising", "jump"])
def test_values_that_climb_along_a_run(kind):
    """A thread's reference moves, and the first chunk's bound is far below the rest."""
    x = torch.randn((3, 120001), device="cuda")
    i = torch.arange(120001, device="cuda")
    x += (i / 200.0 if kind == "rising" else torch.where(i > 90000, 500.0, 0.0))
    tokens = np.array([[0], [120000], [60000]])
    _check(x, 1.0, tokens, 20, _run(x, tokens, 20))
    _check(x.bfloat16(), 1.0, tokens, 20, _run(x.bfloat16(), tokens, 20))
