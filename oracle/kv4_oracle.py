"""CPU oracle of the paged 4-bit cache, its page tables and attention, and of
the token log probabilities: plain numpy, written from the definitions in
include/w12.h, sharing no code with the GPU path. Cache bytes and page tables
are exact (every step is an IEEE fp32 operation or an integer one); attention
and log probabilities are float64."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# Page tables
# ---------------------------------------------------------------------------

OK, ERR_ARG, ERR_WORKSPACE = 0, 1, 3


def pages_update(table, used, free, n_free, start, add, T, page_size):
    """One w12_pages_update on lists of lists / lists (copied): returns
    (table, used, free, n_free, slots [B, T], set of status codes)."""
    table = [list(r) for r in table]
    used, free = list(used), list(free)
    B, max_pages = len(table), len(table[0])
    add = [0] * B if add is None else list(add)
    codes = set()
    slots = [[-1] * T for _ in range(B)]
    served, fits = [], True
    taken = 0
    returned = []
    for b in range(B):
        if start[b] < 0 or add[b] < 0 or add[b] > T or not 0 <= used[b] <= max_pages \
                or start[b] + add[b] > max_pages * page_size:
            codes.add(ERR_ARG)
            continue
        want = -(-(start[b] + add[b]) // page_size)
        grow = want - used[b]
        if grow > 0:
            # In order: the first request that does not fit ends the serving.
            if fits and taken + grow <= n_free:
                for i in range(grow):
                    table[b][used[b] + i] = free[n_free - 1 - (taken + i)]
                taken += grow
            else:
                fits = False
                codes.add(ERR_WORKSPACE)
                continue
        else:
            for i in range(want, used[b]):
                returned.append(table[b][i])
                table[b][i] = -1
        used[b] = want
        served.append(b)
    left = n_free - taken
    for k, page in enumerate(returned):
        free[left + len(returned) - 1 - k] = page
    for b in served:
        for i in range(add[b]):
            pos = start[b] + i
            slots[b][i] = table[b][pos // page_size] * page_size + pos % page_size
    return table, used, free, left + len(returned), slots, codes


# ---------------------------------------------------------------------------
# Rows
# ---------------------------------------------------------------------------

def _bf16(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, round to nearest even; NaN -> 0x7FC0."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32)
    out = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), out)


def _f32(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits).astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantise(x: np.ndarray):
    """Rows x [..., d] (fp32) -> (codes uint8 [..., d] in 0..15, s bits, z bits)."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        r = np.float32(1) / np.float32(15)
        lo, hi = x.min(-1), x.max(-1)
        sb = _bf16(hi * r - lo * r)
        s = _f32(sb)
        tiny = s < np.float32(2.0 ** -100)
        sb, s = np.where(tiny, np.uint16(0), sb), np.where(tiny, np.float32(0), s)
        z = lo + np.float32(8) * s
        # 8 s alone may pass the fp32 range where the sum (one rounding) does not.
        zb = _bf16(np.where(np.isfinite(np.float32(8) * s), z, (lo.astype(np.float64) + 8 * s.astype(np.float64)).astype(np.float32)))
        z = _f32(zb)
        inv = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0)).astype(np.float32)
        q = np.clip(np.rint((x - z[..., None]) * inv[..., None]) + np.float32(8), 0, 15)
        odd = ~np.isfinite(x).all(-1)
        q = np.where(odd[..., None], 8, q).astype(np.uint8)
    return q, np.where(odd, np.uint16(0x7FC0), sb).astype(np.uint16), np.where(odd, np.uint16(0x7FC0), zb).astype(np.uint16)


def values(q: np.ndarray, sb: np.ndarray, zb: np.ndarray) -> np.ndarray:
    """float64 values z + s (q - 8) of code rows [..., d]."""
    with np.errstate(invalid="ignore"):
        return _f32(zb).astype(np.float64)[..., None] + _f32(sb).astype(np.float64)[..., None] * (q.astype(np.float64) - 8)


def row_bytes(q: np.ndarray, r: int) -> np.ndarray:
    """Bytes of one row's codes [d] as they lie in row r of a page."""
    d = len(q)
    out = np.zeros(d // 2, dtype=np.uint8)
    for c in range(d):
        nibble = (c % 8) // 2 + 4 * (c % 2)
        byte = 4 * (c // 8) + nibble // 2
        if d == 128 and (r >> 1) & 1:
            byte ^= 32
        out[byte] |= int(q[c]) << (4 * (nibble % 2))
    return out


def row_codes(b: np.ndarray, r: int) -> np.ndarray:
    """Codes [d] of a row's bytes (the inverse of row_bytes)."""
    d = 2 * len(b)
    q = np.zeros(d, dtype=np.uint8)
    for c in range(d):
        nibble = (c % 8) // 2 + 4 * (c % 2)
        byte = 4 * (c // 8) + nibble // 2
        if d == 128 and (r >> 1) & 1:
            byte ^= 32
        q[c] = (int(b[byte]) >> (4 * (nibble % 2))) & 15
    return q


def _where(P: int, d: int, r: int, which: int):
    """(code bytes, parameter bytes) of row r of K (0) or V (1) within a block."""
    c = (which * P + r) * (d // 2)
    p = P * d + (which * P + r) * 4
    return slice(c, c + d // 2), slice(p, p + 4)


def append(pool: np.ndarray, K, V, slots, d: int) -> np.ndarray:
    """pool [n_pages, Hkv, P (d + 8)] uint8 with rows K, V [n, Hkv, d] (fp32 values) written."""
    pool = pool.copy()
    P = pool.shape[2] // (d + 8)
    for which, x in enumerate((K, V)):
        q, sb, zb = quantise(x)
        for i, slot in enumerate(slots):
            if slot < 0 or slot >= pool.shape[0] * P:
                continue
            r = slot % P
            codes, par = _where(P, d, r, which)
            for h in range(pool.shape[1]):
                pool[slot // P, h, codes] = row_bytes(q[i, h], r)
                pool[slot // P, h, par] = np.array([sb[i, h], zb[i, h]], dtype=np.uint16).view(np.uint8)
    return pool


def read(pool: np.ndarray, slots, d: int):
    """float64 (K, V) [n, Hkv, d] of the given slots (zeros for -1)."""
    n_pages, Hkv, block = pool.shape
    P = block // (d + 8)
    out = np.zeros((2, len(slots), Hkv, d))
    for which in (0, 1):
        for i, slot in enumerate(slots):
            if slot < 0:
                continue
            r = slot % P
            codes, par = _where(P, d, r, which)
            for h in range(Hkv):
                s, z = np.frombuffer(pool[slot // P, h, par].tobytes(), dtype=np.uint16)
                out[which, i, h] = values(row_codes(pool[slot // P, h, codes], r), s, z)
    return out[0], out[1]


def commit(pool: np.ndarray, table, prefix, path, path_len, d: int) -> np.ndarray:
    """pool after the rows prefix + path[b, k] moved to prefix + k (valid paths)."""
    src = pool
    pool = pool.copy()
    P = pool.shape[2] // (d + 8)
    for b in range(len(prefix)):
        for k in range(int(path_len[b])):
            i, j = int(prefix[b]) + int(path[b][k]), int(prefix[b]) + k
            pi, pj = int(table[b][i // P]), int(table[b][j // P])
            for h in range(pool.shape[1]):
                for which in (0, 1):
                    ci, qi = _where(P, d, i % P, which)
                    cj, qj = _where(P, d, j % P, which)
                    pool[pj, h, cj] = row_bytes(row_codes(src[pi, h, ci], i % P), j % P)
                    pool[pj, h, qj] = src[pi, h, qi]
    return pool


# ---------------------------------------------------------------------------
# Attention and log probabilities
# ---------------------------------------------------------------------------

def visible(prefix: int, n: int, parents=None) -> np.ndarray:
    """[n, prefix + n]: whether new token t sees position j."""
    see = np.zeros((n, prefix + n), dtype=bool)
    see[:, :prefix] = True
    for t in range(n):
        if parents is None:
            see[t, prefix:prefix + t + 1] = True
        else:
            i = t
            while i >= 0:
                see[t, prefix + i] = True
                i = int(parents[i])
    return see


def attention(Q, K, V, see, scale):
    """(O, A, eps) of one request: Q [n, Hq, d], K, V [L, Hkv, d] float64, see [n, L].

    O [n, Hq, d] float64; A = sum_j p_j |V_j| and eps = scale max_j |q|.|K_j| over
    the visible keys bound what roundings of the operands can do (see the tests).
    """
    n, Hq, d = Q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    O, A, E = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for h in range(Hq):
        g = h // G
        rows = see.any(0)
        k, v = np.where(rows[:, None], K[:, g], 0), np.where(rows[:, None], V[:, g], 0)
        s = np.where(see, scale * (Q[:, h] @ k.T), -np.inf)
        E[:, h] = np.where(see, scale * (np.abs(Q[:, h]) @ np.abs(k).T), 0).max(1)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        O[:, h] = p @ v
        A[:, h] = p @ np.abs(v)
    return O, A, E


def logprobs(logits: np.ndarray, scale: float, tokens, k: int):
    """(logprob [M, n], entropy [M], lse [M], top_logprob [M, k], top_id [M, k])
    of finite or -inf logits (fp32 values), x = fp32(scale * logit) in float64."""
    x = (np.asarray(logits, dtype=np.float32) * np.float32(scale)).astype(np.float64)
    M, V = x.shape
    tokens = np.asarray(tokens)
    lp = np.zeros(tokens.shape)
    ent, lse = np.zeros(M), np.zeros(M)
    top, ids = np.full((M, k), -np.inf), np.full((M, k), -1, dtype=np.int32)
    for m in range(M):
        row = x[m]
        fin = np.nonzero(row > -np.inf)[0]
        if len(fin) == 0:
            lse[m] = -np.inf
        else:
            mx = row[fin].max()
            e = np.exp(row[fin] - mx)
            lse[m] = mx + np.log(e.sum())
            p = e / e.sum()
            ent[m] = lse[m] - (p * row[fin]).sum()
        for j, t in enumerate(tokens[m]):
            lp[m, j] = 0.0 if t == -1 else -np.inf if row[t] == -np.inf else row[t] - lse[m]
        order = fin[np.argsort(-row[fin], kind="stable")][:k]
        ids[m, :len(order)] = order
        top[m, :len(order)] = row[order] - lse[m]
    return lp, ent, lse, top, ids
