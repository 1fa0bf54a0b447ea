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


def _unchanged(step, b, length, used, table, rows):
    assert int(step.length[b]) == length and int(step.pages.used[b]) == used
    assert torch.equal(step.pages.table[b], table)
    K, V = _rows(step, b, length)
    assert (K == rows[0]).all() and (V == rows[1]).all()


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
