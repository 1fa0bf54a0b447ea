"""The paged verify step (engine.PagedVerifyStep): every part against the oracle on
the values that the step itself produced before it, over several steps."""
import numpy as np
import pytest
import torch

from gpu_util import status_value, to_dev_bf16
from oracle import kv4_oracle as KO
from oracle import w12_oracle as O
from speculative_decoding_verification_w12_gb300 import synthetic as S
from speculative_decoding_verification_w12_gb300 import w12
from speculative_decoding_verification_w12_gb300.engine import PagedVerifyStep

pytestmark = pytest.mark.gpu


def _step(B, T, hidden, Hq, Hkv, d, vocab, **kw):
    W = [S.weights_bf16((Hq + 2 * Hkv) * d, hidden, seed=5), S.weights_bf16(hidden, Hq * d, seed=6),
         S.weights_bf16(vocab, hidden, seed=7)]
    return W, PagedVerifyStep(*(w12.pack(to_dev_bf16(w)) for w in W), B, T, Hq, Hkv, d, **kw)


def test_steps_against_the_oracle():
    B, T, hidden, Hq, Hkv, d, vocab, P = 3, 12, 256, 8, 2, 64, 2048, 16
    W, step = _step(B, T, hidden, Hq, Hkv, d, vocab, n_pages=40, page_size=P, max_len=160, top_k=4)
    g = np.random.default_rng(0)
    prompt = [0, 30, 75]
    kv = g.standard_normal((2, B, 75, Hkv, d)).astype(np.float32)
    dev = [torch.from_numpy(x).cuda() for x in kv]
    step.prefill(dev[0], dev[1], torch.tensor(prompt, dtype=torch.int32, device="cuda"))
    # The oracle's cache of each request: float64 values of its committed rows.
    cached = [[KO.values(*KO.quantise(kv[w, b, :prompt[b]])) for b in range(B)] for w in (0, 1)]
    table = KO.pages_update([[-1] * 10] * B, [0] * B, list(range(39, -1, -1)), 40, [0] * B, prompt, 75, P)
    for n in range(3):
        X = S.activations_bf16(B * T, hidden, seed=50 + n)
        parents = np.stack([S.random_tree(T, max_depth=6, g=g) for _ in range(B)])
        length = step.length.cpu().tolist()
        # A run without acceptance to learn the argmax, then drafts planted on a path of it.
        before = (step.cache.pool.clone(), [t.clone() for t in (step.pages.table, step.pages.used, step.pages.free,
                                                                step.pages.n_free, step.length)])
        args = (to_dev_bf16(X), torch.from_numpy(parents.astype(np.int32)).cuda())
        first = step.run(*args, torch.full((B, T), -1, dtype=torch.int32, device="cuda"))
        assert first["accept_len"].tolist() == [0] * B
        step.cache.pool.copy_(before[0])
        for t, old in zip((step.pages.table, step.pages.used, step.pages.free, step.pages.n_free, step.length), before[1]):
            t.copy_(old)
        draft = g.integers(0, vocab, (B, T)).astype(np.int32)
        draft[:, 1] = first["bonus"].cpu().numpy()          # node 1 is a child of the root
        r = step.run(*args, torch.from_numpy(draft).cuda())
        assert status_value(step.status) == 0
        # Keys, values and queries of the step, from the GPU's own product.
        Y = w12.gemm(args[0], step.qkv).cpu().numpy()
        ref = O.gemm(X, O.pack(W[0]))
        assert np.linalg.norm(Y - ref) <= 1e-3 * np.linalg.norm(ref)
        Y = Y.reshape(B, T, -1)
        out = []
        for b in range(B):
            k, v = (KO.values(*KO.quantise(x.reshape(T, Hkv, d))) for x in
                    (Y[b, :, Hq * d:(Hq + Hkv) * d], Y[b, :, (Hq + Hkv) * d:]))
            q = KO._f32(KO._bf16(Y[b, :, :Hq * d])).astype(np.float64).reshape(T, Hq, d)
            K, V = np.concatenate([cached[0][b], k]), np.concatenate([cached[1][b], v])
            o, _, _ = KO.attention(q, K, V, KO.visible(length[b], T, parents[b]), d ** -0.5)
            out.append(o.reshape(T, -1))
            # Commit: the path's rows follow the committed ones.
            path = r["path"][b, :int(r["path_len"][b])].tolist()
            assert path[0] == 0 and len(path) == int(r["accept_len"][b]) + 1 and len(path) >= 2
            cached[0][b] = np.concatenate([cached[0][b], k[path]])
            cached[1][b] = np.concatenate([cached[1][b], v[path]])
        # Attention, products and logits down to the answered rows: two bf16 roundings
        # (attention output, hidden rows; 2^-8 each) and an fp32 product on the way.
        H = np.stack(out).reshape(B * T, -1) @ KO._f32(W[1]).astype(np.float64).T
        logits = (H @ KO._f32(W[2]).astype(np.float64).T).reshape(B, T, vocab)
        std = logits.std()
        for b in range(B):
            for i, row in enumerate(r["path"][b, :int(r["path_len"][b])].tolist()):
                z = logits[b, row]
                lse = z.max() + np.log(np.exp(z - z.max()).sum())
                tok = int(r["tokens"][b, i])
                tol = 8 * 2.0 ** -8 * std + 1e-4
                assert abs(float(r["logprob"][b, i]) - (z[tok] - lse)) <= tol
                assert abs(float(r["top_logprob"][b, i, 0]) - (z.max() - lse)) <= tol
                assert tok == int(r["top_id"][b, i, 0])              # greedy: the answered token is the likeliest
            assert (r["tokens"][b, int(r["path_len"][b]):] == -1).all()
        # Lengths, pages and the committed rows of the cache.
        now = [length[b] + int(r["path_len"][b]) for b in range(B)]
        assert step.length.cpu().tolist() == now
        assert step.pages.used.cpu().tolist() == [-(-x // P) for x in now]
        t = step.pages.table.cpu().numpy()
        pool = step.cache.pool.cpu().numpy()
        for b in range(B):
            pos = np.arange(now[b])
            K, V = KO.read(pool, (t[b, pos // P] * P + pos % P).tolist(), d)
            assert (K == cached[0][b]).all() and (V == cached[1][b]).all()
    assert table[1] == [-(-x // P) for x in prompt]


def test_example_runs(capsys):
    import os
    import runpy
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_verify.py")
    runpy.run_path(path, run_name="__main__")
    assert capsys.readouterr().out.count("request") == 6


def test_weights_that_do_not_fit_are_refused():
    w = [w12.pack(to_dev_bf16(S.weights_bf16(128, 128, seed=1))) for _ in range(3)]
    with pytest.raises(ValueError):
        PagedVerifyStep(*w, 1, 4, 2, 1, 64, n_pages=4)
