"""PagedVerifyStep's ways in, where a call is not what it should be: prompts whose offsets do not fit their
rows, rows in any layout and type, prompts beside a rotation, adapters of another number of requests. A
request that is refused keeps its state to the byte."""
import numpy as np
import pytest
import torch

from gpu_util import status_value, to_dev_bf16, to_dev_i32
from oracle import kv4_oracle as KO
from oracle import layer_oracle as LO
from speculative_decoding_verification_w12_gb300 import synthetic as S
from speculative_decoding_verification_w12_gb300 import w12
from speculative_decoding_verification_w12_gb300.engine import PagedVerifyStep
from test_gpu_paged_step_layer import B, D, HIDDEN, HKV, HQ, MAX, P, T, VOCAB, _f, _rows, _step

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _plain(n_pages=60):
    """A step that takes queries and keys as they come."""
    W = [S.weights_bf16((HQ + 2 * HKV) * D, HIDDEN, seed=5), S.weights_bf16(HIDDEN, HQ * D, seed=6), S.weights_bf16(VOCAB, HIDDEN, seed=7)]
    return PagedVerifyStep(*(w12.pack(to_dev_bf16(w)) for w in W), B, T, HQ, HKV, D, n_pages=n_pages, page_size=P, max_len=MAX, top_k=2)


def _made(rotated):
    """(step, what its keys become by position)."""
    if rotated:
        step, _, turn_k = _step()
        return step, turn_k
    return _plain(), lambda x, pos: x


def _qkv(n, dtype=F32, seed=1, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((n, h, D), generator=g, device="cuda") * scale).to(dtype) for h in (HQ, HKV, HKV)]


def _state(step):
    p = step.pages
    return [t.clone() for t in (step.length, p.table, p.used, p.n_free, p.free, step.cache.pool)]


def _holds(step, b, k, v):
    """Request b's cached rows are those of the keys k and values v, fp32."""
    for got, want in zip(_rows(step, b, len(k)), (k, v)):
        np.testing.assert_array_equal(got, KO.values(*KO.quantise(want)))


# Offsets, rows, the requests whose prompts are taken.
OFFSETS = [([100, 200, 200, 200], 150, []), ([0, 50, 120, 120], 100, [0]), ([-5, 4, 10, 30], 30, [1, 2]), ([0, -3, 10, 30], 30, [2]),
           ([0, 20, 10, 30], 30, []), ([0, 31, 10, 30], 30, []), ([0, 10, 31, 31], 30, [0]), ([10, 0, 20, 30], 30, [2]), ([-20, -10, 5, 30], 30, [2]),
           ([5, 5, 9, 2 ** 31 - 1], 30, [1]), ([-2 ** 31, 2 ** 31 - 1, 7, 9], 30, []), ([40, 45, 50, 60], 30, []), ([3, 10, 10, 30], 30, [0, 2])]


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("cu,n,taken", OFFSETS, ids=str)
def test_offsets_that_do_not_fit_the_rows(cu, n, taken, rotated):
    """A prompt with a place outside the rows, or that shares rows with another, is not cached; its request
    keeps its length, its pages and what they hold. The others are taken as ever."""
    step, turn = _made(rotated)
    first = [20, 7, 33]
    q, k, v = _qkv(60, seed=2)
    step.prompt(q, k, v, to_dev_i32(np.concatenate([[0], np.cumsum(first)])))
    assert status_value(step.status) == 0
    before, rows = _state(step), [_rows(step, b, x) for b, x in enumerate(first)]
    q, k, v = _qkv(n)
    step.prompt(q, k, v, to_dev_i32(cu))
    good = all(a <= e for a, e in zip(cu, cu[1:])) and cu[0] >= 0 and cu[-1] <= n
    assert status_value(step.status) == (0 if good else 1)
    want = [cu[b + 1] - cu[b] if b in taken else first[b] for b in range(B)]
    assert step.length.tolist() == want
    assert step.pages.used.tolist() == [-(-x // P) for x in want]
    assert int(step.pages.n_free[0]) == 60 - sum(-(-x // P) for x in want)
    for b in range(B):
        if b in taken:
            a, e = cu[b], cu[b + 1]
            _holds(step, b, turn(_f(k[a:e]), np.arange(e - a)), _f(v[a:e]))
        else:
            assert torch.equal(step.pages.table[b], before[1][b])
            for got, old in zip(_rows(step, b, first[b]), rows[b]):
                np.testing.assert_array_equal(got, old)
    if not taken:
        assert all(torch.equal(x, y) for x, y in zip(_state(step), before))


def test_a_step_of_one_request():
    W = [w12.pack(to_dev_bf16(S.weights_bf16(*x, seed=1))) for x in ((512, 128), (128, 256), (1024, 128))]
    step = PagedVerifyStep(*W, 1, 4, 4, 2, D, n_pages=8, page_size=P, max_len=100)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((60, h, D), generator=g, device="cuda") for h in (4, 2, 2))
    for cu, length, code in (([3, 50], 47, 0), ([0, 61], 47, 1), ([-1, 5], 47, 1), ([50, 3], 47, 1), ([7, 7], 47, 0), ([59, 60], 1, 0), ([0, 60], 60, 0)):
        step.status.zero_()
        O = step.prompt(q, k, v, to_dev_i32(cu))
        assert status_value(step.status) == code and step.length.tolist() == [length]
        if code == 0 and cu[1] > cu[0]:
            _holds(step, 0, _f(k[cu[0]:cu[1]]), _f(v[cu[0]:cu[1]]))
            part = [x[cu[0]:cu[1]].bfloat16() for x in (q, k, v)]
            assert torch.equal(O[cu[0]:cu[1]], w12.prompt_attention(*part, to_dev_i32([0, cu[1] - cu[0]])))


def test_a_graph_of_prompts_meets_offsets_that_do_not_fit():
    """Captured with good offsets: replays refuse what an eager call refuses, and serve again."""
    q, k, v = _qkv(90)
    eager, graphed = _plain(), _plain()
    cu = to_dev_i32([0, 30, 60, 90])
    graphed.prompt(q, k, v, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.prompt(q, k, v, cu)
    eager.prompt(q, k, v, cu)
    for offsets in ([0, 50, 20, 90], [0, 10, 40, 91], [-1, 10, 40, 90], [0, 10, 40, 90], [5, 5, 2, 90], [0, 20, 20, 50]):
        for step in (eager, graphed):
            step.status.zero_()
        cu.copy_(to_dev_i32(offsets))
        graph.replay()
        eager.prompt(q, k, v, to_dev_i32(offsets))
        assert status_value(eager.status) == status_value(graphed.status)
        assert torch.equal(eager.length, graphed.length)
        for b, n in enumerate(eager.length.tolist()):
            for x, y in zip(_rows(eager, b, n), _rows(graphed, b, n)):
                np.testing.assert_array_equal(x, y)
    assert graphed.length.tolist() == [20, 30, 30]


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("what", ["type", "type of one", "layout", "host", "offsets"])
def test_rows_that_are_refused_change_nothing(what, rotated):
    step, _ = _made(rotated)
    q, k, v = _qkv(60, seed=2)
    cu = to_dev_i32([0, 20, 27, 60])
    step.prompt(q, k, v, cu)
    torch.cuda.synchronize()
    before = _state(step)
    q, k, v = _qkv(30)
    cu = to_dev_i32([0, 10, 10, 30])                       # fewer pages than the requests have
    if what == "type":
        q, k, v = (x.double() for x in (q, k, v))
    elif what == "type of one":
        v = v.bfloat16()
    elif what == "layout":
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
    elif what == "host":
        v = v.cpu()
    else:
        cu = cu[:3]
    with pytest.raises((ValueError, TypeError)):
        step.prompt(q, k, v, cu)
    assert all(torch.equal(x, y) for x, y in zip(_state(step), before)) and status_value(step.status) == 0


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("how", ["base", "token stride", "head stride"])
def test_rows_at_any_address(how, dtype, rotated):
    """Views that start between 16-byte boundaries, or whose strides are no whole number of them."""
    q, k, v = _qkv(50, dtype)

    def view(x):
        n, h, d = x.shape
        token, head, first = {"base": (h * d, d, 3), "token stride": (h * d + 5, d, 0), "head stride": (h * (d + 1), d + 1, 0)}[how]
        wide = torch.zeros(n * token + 8, dtype=dtype, device="cuda")
        y = wide.as_strided((n, h, d), (token, head, 1), first)
        y.copy_(x)
        return y
    cu, out = to_dev_i32([0, 20, 20, 50]), []
    for rows in ((q, k, v), [view(x) for x in (q, k, v)]):
        step, _ = _made(rotated)
        O = step.prompt(*rows, cu)
        assert status_value(step.status) == 0 and step.length.tolist() == [20, 0, 30]
        out.append((O, _rows(step, 0, 20), _rows(step, 2, 30)))
    assert torch.equal(out[0][0], out[1][0])
    for x, y in zip(out[0][1] + out[0][2], out[1][1] + out[1][2]):
        np.testing.assert_array_equal(x, y)


def test_fp16_prompts_are_attended_over_as_they_are():
    """Without a rotation nothing is rounded on the way to the scores."""
    step = _plain()
    q, k, v = _qkv(120, F16, scale=2.0)
    cu = to_dev_i32([0, 50, 50, 120])
    O = step.prompt(q, k, v, cu)
    assert O.dtype is BF16
    assert torch.equal(O, w12.prompt_attention(q, k, v, cu).to(BF16))


def test_prefill_of_a_step_with_a_rotation():
    """Keys are normed and rotated as those of run() and prompt(); running requests beside them stay."""
    step, _, turn = _step()
    g = torch.Generator(device="cuda").manual_seed(4)
    K, V = (torch.randn((B, 40, HKV, D), generator=g, device="cuda") for _ in range(2))
    step.prefill(K, V, to_dev_i32([40, 0, 13]))
    assert status_value(step.status) == 0 and step.length.tolist() == [40, 0, 13]
    for b, n in ((0, 40), (2, 13)):
        _holds(step, b, turn(_f(K[b, :n]), np.arange(n)), _f(V[b, :n]))
    other = _step()[0]
    rows = [torch.cat([x[0, :40], x[2, :13]]) for x in (K, V)]
    other.prompt(torch.zeros((53, HQ, D), device="cuda"), *rows, to_dev_i32([0, 40, 40, 53]))
    for b, n in ((0, 40), (2, 13)):
        for x, y in zip(_rows(step, b, n), _rows(other, b, n)):
            np.testing.assert_array_equal(x, y)
    step.prefill(K.flip(0), V.flip(0), to_dev_i32([-1, 30, -1]))
    assert status_value(step.status) == 0 and step.length.tolist() == [40, 30, 13]
    _holds(step, 1, turn(_f(K[1, :30]), np.arange(30)), _f(V[1, :30]))
    _holds(step, 0, turn(_f(K[0]), np.arange(40)), _f(V[0]))
    step.status.zero_()
    step.prefill(K, V, to_dev_i32([41, -1, -1]))           # more than the rows
    assert status_value(step.status) == 1 and step.length.tolist() == [40, 30, 13]


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("what", ["type", "type of one", "layout", "host", "heads", "requests", "rows"])
def test_prefilled_rows_that_are_refused_change_nothing(what, rotated):
    step, _ = _made(rotated)
    step.prompt(*_qkv(60, seed=2), to_dev_i32([0, 20, 27, 60]))
    torch.cuda.synchronize()
    before = _state(step)
    K, V = (torch.randn((B, 10, HKV, D), device="cuda") for _ in range(2))
    if what == "type":
        K, V = K.double(), V.double()
    elif what == "type of one":
        V = V.bfloat16()
    elif what == "layout":
        K = K.transpose(2, 3).contiguous().transpose(2, 3)
    elif what == "host":
        V = V.cpu()
    elif what == "heads":
        K, V = K[:, :, :1], V[:, :, :1]
    elif what == "requests":
        K, V = K[:2], V[:2]
    else:
        V = V[:, :9]
    with pytest.raises((ValueError, TypeError)):
        step.prefill(K, V, to_dev_i32([10, 0, 3]))
    assert all(torch.equal(x, y) for x, y in zip(_state(step), before)) and status_value(step.status) == 0


def test_adapters_of_another_number_of_requests_are_refused():
    step = _step()[0]
    step.prompt(*_qkv(60, seed=2), to_dev_i32([0, 20, 27, 60]))
    torch.cuda.synchronize()
    before = _state(step)
    X, tree = torch.zeros((B * T, HIDDEN), dtype=BF16, device="cuda"), to_dev_i32(np.tile(np.arange(-1, T - 1), (B, 1)))
    for bad in (to_dev_i32([1]), to_dev_i32([[1], [0], [2]]), to_dev_i32([0, 1]), to_dev_i32([0, 1, 2, 0]), to_dev_i32([0, 1, 2]).long(),
                torch.zeros(B, dtype=torch.int32), torch.zeros((), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            step.run(X, tree, torch.zeros_like(tree), adapter=bad)
        assert all(torch.equal(x, y) for x, y in zip(_state(step), before)) and status_value(step.status) == 0
    # A strided one of the right number is as good as any.
    wide = to_dev_i32([[2, 9], [-1, 9], [0, 9]])
    a, b = (_step()[0].run(X + 1, tree, torch.zeros_like(tree), adapter=x) for x in (wide[:, 0], wide[:, 0].contiguous()))
    assert all(torch.equal(a[k], b[k]) for k in a)
