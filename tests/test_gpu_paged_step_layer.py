"""The paged verify step with everything between its products: prompts admitted and attended over,
heads normed and rotated, adapters beside the products; each part against the oracle on the values
that the step itself produced before it, as a graph too."""
import numpy as np
import pytest
import torch

from gpu_util import status_value, to_dev_bf16, to_dev_i32
from oracle import kv4_oracle as KO
from oracle import layer_oracle as LO
from speculative_decoding_verification_w12_gb300 import synthetic as S
from speculative_decoding_verification_w12_gb300 import w12
from speculative_decoding_verification_w12_gb300.engine import PagedVerifyStep

pytestmark = pytest.mark.gpu
B, T, HIDDEN, HQ, HKV, D, VOCAB, P, MAX = 3, 12, 256, 8, 2, 64, 1024, 16, 200


def _adapters(N, K, seed, n=3, rank=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A, Bm = (torch.randn(s, generator=g, device="cuda") * 0.03 for s in ((n, rank, K), (n, N, rank)))
    return w12.LoRA(A.bfloat16(), Bm.bfloat16(), torch.rand(n, generator=g, device="cuda") + 0.5)


def _step(n_pages=60, adapters=True, pairs=False):
    W = [S.weights_bf16((HQ + 2 * HKV) * D, HIDDEN, seed=5), S.weights_bf16(HIDDEN, HQ * D, seed=6), S.weights_bf16(VOCAB, HIDDEN, seed=7)]
    g = np.random.default_rng(3)
    qw, kw = (g.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    tab = LO.table(MAX, 32)
    rope = w12.Rope(torch.from_numpy(tab).cuda(), D, torch.from_numpy(qw).cuda(), torch.from_numpy(kw).cuda(), 1e-6, pairs)
    some = {"qkv": _adapters((HQ + 2 * HKV) * D, HIDDEN, 1), "out": _adapters(HIDDEN, HQ * D, 2), "head": _adapters(VOCAB, HIDDEN, 4)}
    step = PagedVerifyStep(*(w12.pack(to_dev_bf16(w)) for w in W), B, T, HQ, HKV, D, n_pages=n_pages, page_size=P, max_len=MAX, top_k=2,
                           rope=rope, adapters=some if adapters else None)

    def turned(x, w, pos):
        return LO.rope(x, w, 1e-6, pos, tab, pairs)
    return step, lambda x, pos: turned(x, qw, pos), lambda x, pos: turned(x, kw, pos)


def _rows(step, b, n):
    t = step.pages.table[b].cpu().numpy()
    pos = np.arange(n)
    return KO.read(step.cache.pool.cpu().numpy(), (t[pos // P] * P + pos % P).tolist(), D)


def _f(t):
    return t.float().cpu().numpy()


def _bf16(x):
    return KO._f32(KO._bf16(x)).astype(np.float64)


@pytest.mark.parametrize("pairs", [False, True])
def test_prompts_then_steps(pairs):
    step, turn_q, turn_k = _step(pairs=pairs)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [40, 0, 75]
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1]) + 5                                   # rows behind the last prompt are nobody's
    wide = torch.randn((n, (HQ + 2 * HKV) * D), generator=g, device="cuda")
    Q, K, V = (x.unflatten(1, (-1, D)) for x in wide.split([HQ * D, HKV * D, HKV * D], 1))
    O = step.prompt(Q, K, V, to_dev_i32(cu))
    assert status_value(step.status) == 0 and step.length.tolist() == lens and O.dtype is torch.bfloat16
    pos = np.concatenate([np.arange(x) for x in lens] + [[-1] * 5])
    k = turn_k(_f(K), pos)
    o, a, e, _ = LO.prompt_attention(_bf16(turn_q(_f(Q), pos)), _bf16(k), _bf16(_f(V)), cu, D ** -0.5)
    # Weights and outputs round to bf16 (2^-8 each); a query's own rounding may fall to the other side
    # of its border (2^-8 of it): scores off by 2^-8 e, weights by twice that.
    m = int(cu[-1])
    tol = 2.0 ** -8 * (np.abs(o) + 1.02 * a) + 2 * 2.0 ** -8 * e[..., None] * a + 2.0 ** -18 * a
    assert (np.abs(_f(O)[:m] - o[:m]) <= tol[:m]).all()
    cached = {}
    for b, x in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        want = [KO.values(*KO.quantise(y[rows])) for y in (k, _f(V))]
        got = _rows(step, b, x)
        assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
        cached[b] = want
    adapter = [2, -1, 0]
    ids = np.repeat(adapter, T)
    for i in range(2):
        X = to_dev_bf16(S.activations_bf16(B * T, HIDDEN, seed=50 + i))
        parents = np.stack([S.random_tree(T, max_depth=6, g=np.random.default_rng(9 + i)) for _ in range(B)])
        length = step.length.tolist()
        draft = np.random.default_rng(i).integers(0, VOCAB, (B, T)).astype(np.int32)
        before = step.cache.pool.clone(), [t.clone() for t in (step.pages.table, step.pages.used, step.pages.free, step.pages.n_free, step.length)]
        args = X, to_dev_i32(parents)
        first = step.run(*args, to_dev_i32(np.full((B, T), -1)), adapter=to_dev_i32(adapter))
        step.cache.pool.copy_(before[0])
        for t, old in zip((step.pages.table, step.pages.used, step.pages.free, step.pages.n_free, step.length), before[1]):
            t.copy_(old)
        draft[:, 1] = first["bonus"].cpu().numpy()        # node 1 is a child of the root: accepted
        r = step.run(*args, to_dev_i32(draft), adapter=to_dev_i32(adapter))
        assert status_value(step.status) == 0 and (r["accept_len"] >= 1).all()
        # The first product with its adapters, then keys, values and queries from the GPU's own.
        lora = step.adapters["qkv"]
        base = w12.gemm(X, step.qkv)
        Y = base.clone()
        lora.run(X, Y, to_dev_i32(ids))
        want, most = LO.lora(_f(X), _f(base), _f(lora.A), _f(lora.B), _f(lora.scale), ids)
        assert (np.abs(_f(Y) - want) <= 7 * 2.0 ** -20 * most + 2.0 ** -24 * np.abs(want)).all()
        Y = _f(Y).reshape(B, T, -1)
        at = LO.tree_positions(length, parents, None, T)
        logits = []
        for b in range(B):
            q, k, v = (x.reshape(T, -1, D) for x in np.split(Y[b], [HQ * D, (HQ + HKV) * D], 1))
            kq, vq = (KO.values(*KO.quantise(x)) for x in (turn_k(k, at[b]), v))
            K, V = (np.concatenate([c, x]) for c, x in zip(cached[b], (kq, vq)))
            o, _, _ = KO.attention(_bf16(turn_q(q, at[b])), K, V, KO.visible(length[b], T, parents[b]), D ** -0.5)
            path = r["path"][b, :int(r["path_len"][b])].tolist()
            cached[b] = [np.concatenate([c, x[path]]) for c, x in zip(cached[b], (kq, vq))]
            x = _bf16(o.reshape(T, -1))
            for name, w in (("out", step.out), ("head", step.head)):
                y = x @ _f(w12.unpack(w)).astype(np.float64).T
                lo = step.adapters[name]
                y = LO.lora(x, y, _f(lo.A), _f(lo.B), _f(lo.scale), [adapter[b]] * T)[0]
                x = _bf16(y)
            logits.append(y)
        std = np.std(logits)
        for b in range(B):
            for j, row in enumerate(r["path"][b, :int(r["path_len"][b])].tolist()):
                z = logits[b][row]
                lse = z.max() + np.log(np.exp(z - z.max()).sum())
                tok = int(r["tokens"][b, j])
                # Three roundings to bf16 on the way (queries, attention output, hidden rows: 2^-8 each).
                assert abs(float(r["logprob"][b, j]) - (z[tok] - lse)) <= 10 * 2.0 ** -8 * std + 1e-4
            now = length[b] + int(r["path_len"][b])
            K, V = _rows(step, b, now)
            assert (K == cached[b][0]).all() and (V == cached[b][1]).all()
            assert int(step.length[b]) == now


def test_a_graph_of_the_step_gives_the_same():
    X = to_dev_bf16(S.activations_bf16(B * T, HIDDEN, seed=50))
    parents, draft = to_dev_i32(np.stack([np.arange(-1, T - 1)] * B)), to_dev_i32(np.zeros((B, T)))
    adapter = to_dev_i32([1, 1, -1])
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn((100, h, D), generator=g, device="cuda") for h in (HQ, HKV, HKV)]
    out = []
    for captured in (False, True):
        step = _step()[0]
        step.prompt(*rows, to_dev_i32([0, 30, 30, 100]))
        assert step.length.tolist() == [30, 0, 70]
        if captured:
            step.run(X, parents, draft, adapter=adapter)  # warm
            step = _step()[0]
            step.prompt(*rows, to_dev_i32([0, 30, 30, 100]))
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                r = step.run(X, parents, draft, adapter=adapter)
            graph.replay()
        else:
            r = step.run(X, parents, draft, adapter=adapter)
        torch.cuda.synchronize()
        assert status_value(step.status) == 0
        out.append({k: v.clone() for k, v in r.items()} | {"length": step.length.clone()})
    for k in out[0]:
        assert torch.equal(out[0][k], out[1][k]), k


def test_prompts_that_do_not_fit_leave_their_requests_as_they_were():
    step = _step(n_pages=6)[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn((150, h, D), generator=g, device="cuda") for h in (HQ, HKV, HKV)]
    O = step.prompt(*rows, to_dev_i32([0, 20, 20, 140]))   # the last needs 8 pages where 4 are left
    assert status_value(step.status) == 3 and step.length.tolist() == [20, 0, 0]
    want = step.rope.run(rows[0], rows[1], to_dev_i32(np.concatenate([np.arange(20), np.arange(120), [-1] * 10])))
    ref = w12.prompt_attention(*want, rows[2].bfloat16(), to_dev_i32([0, 20, 20, 140]))
    assert torch.equal(O[:140], ref[:140])
    step.status.zero_()
    step.prompt(*(x[:30] for x in rows), to_dev_i32([0, 0, 30, 30]))
    assert status_value(step.status) == 0 and step.length.tolist() == [20, 30, 0]
    step.status.zero_()
    step.prompt(*rows, to_dev_i32([0, 0, 0, 150]), longest=100)
    assert status_value(step.status) == 1 and step.length.tolist() == [20, 30, 0]


def test_parts_that_do_not_fit_are_refused():
    W = [w12.pack(to_dev_bf16(S.weights_bf16(*s, seed=1))) for s in ((512, 128), (128, 256), (1024, 128))]
    args = (*W, 1, 4, 4, 2, 64)
    PagedVerifyStep(*args, n_pages=4, max_len=64)
    for bad in (dict(rope=w12.Rope.create(128, 64)), dict(rope=w12.Rope.create(64, 63)), dict(adapters={"mlp": _adapters(512, 128, 1)}),
                dict(adapters={"qkv": _adapters(128, 256, 1)})):
        with pytest.raises(ValueError):
            PagedVerifyStep(*args, n_pages=4, max_len=64, **bad)


def test_prompts_and_adapters_that_the_step_refuses():
    step = _step(adapters=False)[0]
    Q, K, V = (torch.randn((30, h, D), device="cuda") for h in (HQ, HKV, HKV))
    cu = to_dev_i32([0, 30, 30, 30])
    for bad in ((Q, K, V, cu.long()), (Q, K, V, cu[:3]), (Q[:29], K, V, cu), (Q, K, V[:29], cu), (K, K, V, cu), (Q, K, V.bfloat16(), cu)):
        with pytest.raises(ValueError):
            step.prompt(*bad)
    assert step.length.tolist() == [0, 0, 0] and status_value(step.status) == 0
    X, tree = torch.zeros((B * T, HIDDEN), dtype=torch.bfloat16, device="cuda"), to_dev_i32(np.tile(np.arange(-1, T - 1), (B, 1)))
    with pytest.raises(ValueError):
        step.run(X, tree, torch.zeros_like(tree), adapter=to_dev_i32([0, 0, 0]))
    W = [w12.pack(to_dev_bf16(S.weights_bf16(*s, seed=1))) for s in ((512, 128), (128, 256), (1024, 128))]
    few = w12.LoRA(*(torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 8, 128), (1, 512, 8))), torch.ones(1, device="cuda"), max_rows=7)
    with pytest.raises(ValueError):
        PagedVerifyStep(*W, 2, 4, 4, 2, 64, n_pages=4, max_len=64, adapters={"qkv": few})


def test_no_prompts_at_all():
    step = _step()[0]
    none = [torch.empty((0, h, D), device="cuda") for h in (HQ, HKV, HKV)]
    assert step.prompt(*none, to_dev_i32([0, 0, 0, 0])).shape == (0, HQ, D)
    torch.cuda.synchronize()
    assert step.length.tolist() == [0, 0, 0] and status_value(step.status) == 0 and not step.pages.used.any()


def test_a_graph_of_prompts_takes_other_offsets():
    """Captured with one set of prompts, replayed with others of as many rows; eager beside it."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rows = [torch.randn((90, h, D), generator=g, device="cuda") for h in (HQ, HKV, HKV)]
    eager, graphed = (_step()[0] for _ in range(2))
    cu = to_dev_i32([0, 30, 60, 90])
    graphed.prompt(*rows, cu)          # (makes what is made once)
    graphed.pages.trim(torch.zeros_like(graphed.length))
    graphed.length.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.prompt(*rows, cu)
    for offsets in ([0, 90, 90, 90], [0, 1, 2, 77], [0, 0, 45, 90]):
        for step in (eager, graphed):
            step.pages.trim(torch.zeros_like(step.length))
            step.length.zero_()
        cu.copy_(to_dev_i32(offsets))
        graph.replay()
        want = eager.prompt(*rows, to_dev_i32(offsets))
        n = offsets[-1]
        assert torch.equal(out[:n], want[:n]) and torch.equal(graphed.length, eager.length)
        assert graphed.length.tolist() == np.diff(offsets).tolist()
        for b, k in enumerate(np.diff(offsets)):
            for x, y in zip(_rows(graphed, b, int(k)), _rows(eager, b, int(k))):
                np.testing.assert_array_equal(x, y)
    assert status_value(graphed.status) == 0 and status_value(eager.status) == 0


def test_without_launch_overlap():
    """Launches that wait for one another give the same bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = [torch.randn((60, h, D), generator=g, device="cuda") for h in (HQ, HKV, HKV)]
    X = torch.randn((B * T, HIDDEN), generator=g, device="cuda").bfloat16()
    tree = to_dev_i32(np.tile(np.arange(-1, T - 1), (B, 1)))
    draft, which = torch.zeros_like(tree), to_dev_i32([0, -1, 2])
    got = []
    for overlap in (True, False):
        step = _step()[0]
        w12.set_overlap(overlap)
        try:
            O = step.prompt(*rows, to_dev_i32([0, 20, 40, 60]))
            r = step.run(X, tree, draft, adapter=which)
            torch.cuda.synchronize()
        finally:
            w12.set_overlap(True)
        assert status_value(step.status) == 0
        got.append([O, step.length] + [r[k] for k in sorted(r)])
    assert all(torch.equal(x, y) for x, y in zip(*got))
