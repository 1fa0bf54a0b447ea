"""The paged verify step (engine.PagedVerifyStep) at its limits: too few pages, a request
at the end of its context, prompts admitted beside running requests, and the step as a
graph."""
import numpy as np
import pytest
import torch

from gpu_util import status_value, to_dev_bf16, to_dev_i32
from oracle import kv4_oracle as KO
from speculative_decoding_verification_w12_gb300 import synthetic as S
from speculative_decoding_verification_w12_gb300 import w12
from speculative_decoding_verification_w12_gb300.engine import PagedVerifyStep

pytestmark = pytest.mark.gpu

T, HIDDEN, HQ, HKV, D, VOCAB, P = 12, 256, 8, 2, 64, 1024, 16


def _step(B, n_pages, max_len, top_k=2):
    W = [S.weights_bf16((HQ + 2 * HKV) * D, HIDDEN, seed=5), S.weights_bf16(HIDDEN, HQ * D, seed=6),
         S.weights_bf16(VOCAB, HIDDEN, seed=7)]
    return PagedVerifyStep(*(w12.pack(to_dev_bf16(w)) for w in W), B, T, HQ, HKV, D, n_pages=n_pages, page_size=P,
                           max_len=max_len, top_k=top_k)


def _prompt(g, B, n):
    kv = g.standard_normal((2, B, n, HKV, D)).astype(np.float32)
    return kv, [torch.from_numpy(x).cuda() for x in kv]


def _inputs(B, n):
    g = np.random.default_rng(100 + n)
    parents = np.stack([S.random_tree(T, max_depth=6, g=g) for _ in range(B)]).astype(np.int32)
    draft = g.integers(0, VOCAB, (B, T)).astype(np.int32)
    return to_dev_bf16(S.activations_bf16(B * T, HIDDEN, seed=60 + n)), to_dev_i32(parents), to_dev_i32(draft)


def _rows(step, b, n):
    """Float64 K and V of request b's first n cached rows."""
    t = step.pages.table[b].cpu().numpy()
    pos = np.arange(n)
    return KO.read(step.cache.pool.cpu().numpy(), (t[pos // P] * P + pos % P).tolist(), D)


def _same_as_alone(step, r, b, before, x):
    """Request b's results are those of a step in which only it takes part."""
    other = _step(1, 64, 1024)
    for name in ("tokens", "path", "accept_len", "bonus"):
        assert r[name].shape[0] == step.B
    K, V = before
    other.prefill(torch.from_numpy(K[None].astype(np.float32)).cuda(), torch.from_numpy(V[None].astype(np.float32)).cuda(),
                  to_dev_i32([K.shape[0]]))
    kk, vv = _rows(other, 0, K.shape[0])
    if not ((kk == K).all() and (vv == V).all()):
        return                                         # (codes do not always quantise to themselves)
    X, parents, draft = x
    q = other.run(X[b * T:(b + 1) * T].contiguous(), parents[b:b + 1].contiguous(), draft[b:b + 1].contiguous())
    for name in ("tokens", "path", "accept_len", "bonus"):
        assert torch.equal(q[name][0], r[name][b]), name


def _unchanged(step, b, length, used, table, rows):
    assert int(step.length[b]) == length and int(step.pages.used[b]) == used
    assert torch.equal(step.pages.table[b], table)
    K, V = _rows(step, b, length)
    assert (K == rows[0]).all() and (V == rows[1]).all()


def _not_served(r, b):
    assert int(r["accept_len"][b]) == 0 and int(r["path_len"][b]) == 0 and int(r["bonus"][b]) == -1
    assert (r["tokens"][b] == -1).all() and (r["path"][b] == -1).all()


def test_a_request_without_pages_keeps_its_state():
    """Three requests of which the second and third need a page that is not there."""
    B, prompt = 3, [20, 28, 30]
    step = _step(B, n_pages=6, max_len=256)
    g = np.random.default_rng(1)
    _, dev = _prompt(g, B, 30)
    step.prefill(*dev, to_dev_i32(prompt))
    assert status_value(step.status) == 0 and int(step.pages.n_free[0]) == 0
    before = [_rows(step, b, n) for b, n in enumerate(prompt)]
    tables, used = step.pages.table.clone(), step.pages.used.tolist()
    x = _inputs(B, 0)
    r = step.run(*x)
    assert status_value(step.status) == 3
    assert int(r["path_len"][0]) == int(r["accept_len"][0]) + 1 and int(step.length[0]) == 20 + int(r["path_len"][0])
    _same_as_alone(step, r, 0, before[0], x)
    for b in (1, 2):
        _not_served(r, b)
        _unchanged(step, b, prompt[b], used[b], tables[b], before[b])
    # Pages that come back serve it: the first request ends.
    step.status.zero_()
    step.prefill(dev[0], dev[1], to_dev_i32([0, -1, -1]))
    r = step.run(*x)
    assert int(step.length[0]) <= T and status_value(step.status) in (0, 3)
    assert int(r["path_len"][1]) >= 1 and int(step.length[1]) == 28 + int(r["path_len"][1])


@pytest.mark.parametrize("max_len", [64, 60, 50])
def test_a_request_at_the_end_of_its_context(max_len):
    """The second request's tokens would pass max_len, which need not be whole pages."""
    B, prompt = 2, [10, max_len - T + 1]
    step = _step(B, n_pages=32, max_len=max_len)
    g = np.random.default_rng(2)
    _, dev = _prompt(g, B, prompt[1])
    step.prefill(*dev, to_dev_i32(prompt))
    assert status_value(step.status) == 0
    before = [_rows(step, b, n) for b, n in enumerate(prompt)]
    used, tables = step.pages.used.tolist(), step.pages.table.clone()
    x = _inputs(B, 1)
    r = step.run(*x)
    assert status_value(step.status) == 1
    _not_served(r, 1)
    _unchanged(step, 1, prompt[1], used[1], tables[1], before[1])
    assert int(step.length[0]) == 10 + int(r["path_len"][0])
    _same_as_alone(step, r, 0, before[0], x)


def test_a_request_just_inside_its_context_is_served():
    step = _step(1, n_pages=8, max_len=50)
    _, dev = _prompt(np.random.default_rng(3), 1, 50 - T)
    step.prefill(*dev, to_dev_i32([50 - T]))
    r = step.run(*_inputs(1, 2))
    assert status_value(step.status) == 0 and int(step.length[0]) == 50 - T + int(r["path_len"][0])


def test_prompts_admitted_beside_running_requests():
    B = 3
    step = _step(B, n_pages=32, max_len=256)
    g = np.random.default_rng(4)
    _, dev = _prompt(g, B, 40)
    step.prefill(*dev, to_dev_i32([17, 0, 40]))
    step.run(*_inputs(B, 3))
    length = step.length.tolist()
    before = [_rows(step, b, n) for b, n in enumerate(length)]
    tables, used = step.pages.table.clone(), step.pages.used.tolist()
    kv, dev = _prompt(g, B, 33)
    step.prefill(*dev, to_dev_i32([-1, 33, -1]))
    assert status_value(step.status) == 0
    for b in (0, 2):
        _unchanged(step, b, length[b], used[b], tables[b], before[b])
    assert int(step.length[1]) == 33 and int(step.pages.used[1]) == 3
    K, V = _rows(step, 1, 33)
    assert (K == KO.values(*KO.quantise(kv[0, 1]))).all() and (V == KO.values(*KO.quantise(kv[1, 1]))).all()
    # Ended by a prompt of no tokens: its pages are free again.
    free = int(step.pages.n_free[0])
    step.prefill(dev[0], dev[1], to_dev_i32([-1, 0, -1]))
    assert int(step.length[1]) == 0 and int(step.pages.n_free[0]) == free + 3
    _unchanged(step, 0, length[0], used[0], tables[0], before[0])


def test_prompts_that_do_not_fit_leave_their_requests_as_they_were():
    B = 2
    step = _step(B, n_pages=4, max_len=60)
    g = np.random.default_rng(5)
    _, dev = _prompt(g, B, 61)
    step.prefill(*dev, to_dev_i32([20, 9]))
    before = [_rows(step, b, n) for b, n in enumerate([20, 9])]
    tables, used = step.pages.table.clone(), step.pages.used.tolist()
    for prompt, code in (([-1, 50], 3), ([61, -1], 1)):            # more pages than are free; past max_len
        step.status.zero_()
        step.prefill(*dev, to_dev_i32(prompt))
        assert status_value(step.status) == code
        for b, n in enumerate([20, 9]):
            _unchanged(step, b, n, used[b], tables[b], before[b])


def test_the_step_as_a_graph():
    """Captured once and replayed, the step answers as eager steps do."""
    B, prompt = 2, [33, 70]
    g = np.random.default_rng(6)
    _, dev = _prompt(g, B, 70)
    eager, graph = _step(B, 40, 256), _step(B, 40, 256)
    for s in (eager, graph):
        s.prefill(*dev, to_dev_i32(prompt))
    x = [t.clone() for t in _inputs(B, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [graph.cache.pool, graph.pages.table, graph.pages.used, graph.pages.free, graph.pages.n_free, graph.length]
    with torch.cuda.stream(side):                      # warm-up, taken back below
        kept = [t.clone() for t in state]
        graph.run(*x)
        for t, k in zip(state, kept):
            t.copy_(k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        out = graph.run(*x)
    for n in range(3):
        for t, new in zip(x, _inputs(B, 5 + n)):
            t.copy_(new)
        want = eager.run(*x)
        cg.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(want[name], out[name]), (n, name)
        assert torch.equal(eager.length, graph.length) and torch.equal(eager.cache.pool, graph.cache.pool)
    assert status_value(eager.status) == 0 and status_value(graph.status) == 0
