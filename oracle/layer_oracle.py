"""CPU oracle of what a layer does between its products: norms of heads with the rotation by
position, positions of draft trees, causal attention over packed prompts, low-rank adapters.
Plain numpy from the definitions in include/w12.h, sharing no code with the GPU path. Rotated
rows are exact fp32 (each step is an IEEE operation); attention and adapters are float64."""
from __future__ import annotations

import numpy as np


def table(max_pos: int, rot_dim: int, theta: float = 10000.0) -> np.ndarray:
    """fp32 [max_pos, rot_dim]: cosines of a position's angles, then their sines."""
    a = np.arange(max_pos, dtype=np.float64)[:, None] * theta ** (-np.arange(0, rot_dim, 2) / rot_dim)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rope(x, weight, eps, positions, tab, interleaved=False) -> np.ndarray:
    """fp32 rows [n, H, d] of fp32 values x, normed (weight not None) and rotated; rows of
    positions outside the table are zeros."""
    x = np.asarray(x, dtype=np.float32)
    if weight is not None:
        with np.errstate(all="ignore"):
            mean = np.square(x.astype(np.float64)).mean(-1, keepdims=True)
            r = (1.0 / np.sqrt(mean + np.float64(np.float32(eps)))).astype(np.float32)
            x = (x * r) * np.asarray(weight, dtype=np.float32)
    positions, rot = np.asarray(positions), tab.shape[1]
    there = (positions >= 0) & (positions < len(tab))
    row = tab[np.where(there, positions, 0)][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out = x.copy()
    with np.errstate(all="ignore"):
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    out[~there] = 0
    return out


def tree_positions(prefix, parents, q_len, T):
    """Positions [B][T] of valid trees (parents None: the order of the tokens)."""
    out = np.full((len(prefix), T), -1, dtype=np.int64)
    for b, a in enumerate(prefix):
        for t in range(T if q_len is None else int(q_len[b])):
            depth, i = t, t
            if parents is not None:
                depth = 0
                while parents[b][i] >= 0:
                    i, depth = int(parents[b][i]), depth + 1
            out[b, t] = a + depth
    return out


def prompt_attention(Q, K, V, cu, scale):
    """(O, A, E, S) of packed prompts in float64: O [total, Hq, d] (NaN outside the sequences),
    and what bounds the kernel's roundings: A = sum_j p_j |V_j|, E [total, Hq] the largest
    scale |q|.|K_j|, S = sum_j |V_j| over the keys seen."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    Hq, Hkv = Q.shape[1], K.shape[1]
    O, A, S = (np.full(Q.shape, np.nan) for _ in range(3))
    E = np.full(Q.shape[:2], np.nan)
    for a, e in zip(cu[:-1], cu[1:]):
        n = int(e) - int(a)
        if n <= 0:
            continue
        see = np.tril(np.ones((n, n), dtype=bool))
        for h in range(Hq):
            q, k, v = Q[a:e, h], K[a:e, h * Hkv // Hq], V[a:e, h * Hkv // Hq]
            s = np.where(see, scale * (q @ k.T), -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            O[a:e, h], A[a:e, h], S[a:e, h] = p @ v, p @ np.abs(v), np.cumsum(np.abs(v), 0)
            E[a:e, h] = np.where(see, scale * (np.abs(q) @ np.abs(k).T), 0).max(1)
    return O, A, E, S


def lora(X, Y, A, B, scale, ids):
    """(Y + adapters, bound) in float64; bound = scale |B| (|A| |x|), what roundings are relative to."""
    out, most = np.asarray(Y, dtype=np.float64).copy(), np.zeros(np.shape(Y))
    for m, a in enumerate(ids):
        if a >= 0:
            x, wa, wb, s = (np.asarray(v, dtype=np.float64) for v in (X[m], A[a], B[a], scale[a]))
            out[m] += s * (wb @ (wa @ x))
            most[m] = abs(s) * (np.abs(wb) @ (np.abs(wa) @ np.abs(x)))
    return out, most
