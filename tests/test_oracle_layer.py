"""Pins of the oracle of rotation, tree positions, prompt attention and adapters: hand values,
closed forms and other ways to the same numbers."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as KO
from oracle import layer_oracle as O


def test_table_by_hand():
    t = O.table(3, 16, theta=100.0)
    assert t.dtype == np.float32 and t.shape == (3, 16)
    assert (t[0] == [1] * 8 + [0] * 8).all()
    assert t[2, 0] == np.float32(np.cos(2.0)) and t[2, 8] == np.float32(np.sin(2.0))
    assert t[1, 4] == np.float32(np.cos(0.1)) and t[2, 12] == np.float32(np.sin(0.2))   # 100^(-8/16) = 0.1


def test_far_positions_keep_their_angles():
    t = O.table(70000, 16)
    a = 69999 - 2 * np.pi * np.floor(69999 / (2 * np.pi))
    assert abs(t[69999, 0] - np.cos(a)) < 1e-7 + 1e-10


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product(pairs):
    g = np.random.default_rng(0)
    x, pos, t = g.standard_normal((5, 2, 64)).astype(np.float32), np.array([0, 1, 7, 30, 31]), O.table(32, 32)
    y = O.rope(x, None, 0.0, pos, t, pairs).astype(np.float64)
    i, j = (slice(0, 32, 2), slice(1, 32, 2)) if pairs else (slice(0, 16), slice(16, 32))
    z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(16) / 16))[:, None]
    assert np.abs(y[..., i] - z.real).max() < 1e-6 and np.abs(y[..., j] - z.imag).max() < 1e-6
    assert (y[..., 32:] == x[..., 32:]).all() and (y[0] == x[0]).all()


def test_scores_depend_on_the_distance():
    g = np.random.default_rng(1)
    q, k, t = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64)), O.table(200, 64)
    dot = lambda a, b: float((O.rope(q, None, 0, [a], t) * O.rope(k, None, 0, [b], t)).sum())  # noqa: E731
    assert abs(dot(50, 20) - dot(180, 150)) < 1e-4 < abs(dot(50, 20) - dot(50, 21))


def test_norm_by_hand():
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[..., :2] = [3, 4]
    w = np.arange(64, dtype=np.float32)
    y = O.rope(x, w, 1e-6, [0], O.table(1, 16))
    assert y[0, 0, 1] == np.float32(4) * np.float32(1 / np.sqrt(25 / 64 + np.float64(np.float32(1e-6))))
    assert y[0, 0, 0] == 0 and (y[0, 0, 2:] == 0).all()
    assert (O.rope(x, w, 1e-6, [-1], O.table(1, 16)) == 0).all() and (O.rope(x, w, 1e-6, [1], O.table(1, 16)) == 0).all()


def test_positions_of_a_hand_tree_and_a_chain():
    tree = [[-1, 0, 0, 1, 3, 2]]
    assert O.tree_positions([10], tree, None, 6).tolist() == [[10, 11, 11, 12, 13, 12]]
    assert O.tree_positions([10], tree, [4], 6).tolist() == [[10, 11, 11, 12, -1, -1]]
    chain = [[-1, 0, 1, 2]]
    assert (O.tree_positions([5], chain, None, 4) == O.tree_positions([5], None, None, 4)).all()


def test_prompt_attention_against_the_other_oracle_and_the_library():
    g = np.random.default_rng(2)
    cu = [0, 5, 5, 6, 20]
    Q, K, V = (g.standard_normal((22, h, 64)) for h in (4, 2, 2))
    o, a, e, s = O.prompt_attention(Q, K, V, cu, 0.2)
    assert np.isnan(o[20:]).all() and np.isfinite(o[:20]).all()
    for b in range(4):
        x = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        if n:
            want, bound, _ = KO.attention(Q[x], K[x], V[x], KO.visible(0, n), 0.2)
            assert np.abs(o[x] - want).max() < 1e-12 and np.abs(a[x] - bound).max() < 1e-12
            t = [torch.from_numpy(np.repeat(y[x], 4 // y.shape[1], 1)).transpose(0, 1) for y in (Q, K, V)]
            lib = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True, scale=0.2).transpose(0, 1)
            assert np.abs(o[x] - lib.numpy()).max() < 1e-12
    assert (o[5] == V[5].repeat(2, 0)).all() and (s >= a - 1e-12)[:20].all() and (e[:20] > 0).all()


def test_adapters_by_hand():
    A, B = np.zeros((2, 8, 16)), np.zeros((2, 16, 8))
    A[1, 3, 5], B[1, 7, 3] = 2.0, -4.0
    X, Y = np.zeros((3, 16)), np.ones((3, 16))
    X[:, 5] = [1, 3, 5]
    out, most = O.lora(X, Y, A, B, [10.0, 0.5], [1, -1, 0])
    assert out[0, 7] == 1 - 4 and most[0, 7] == 4 and (np.delete(out.ravel(), 7) == 1).all()
