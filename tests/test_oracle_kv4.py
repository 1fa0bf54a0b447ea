"""Pins of the 4-bit cache's oracle, and the host checks of its entry points
(no GPU needed)."""
import ctypes

import numpy as np
import pytest

from oracle import kv4_oracle as O
from speculative_decoding_verification_w12_gb300 import build as B
from speculative_decoding_verification_w12_gb300 import w12


@pytest.fixture(scope="module")
def L():
    B.build()
    return w12.lib()


# ------------------------------------------------------------------ oracle
def test_quantiser_by_hand():
    # min 0, max 15: s = 1, z = 8, codes are the values themselves.
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :16] = np.arange(16)
    q, s, z = O.quantise(x)
    assert O._f32(s)[0] == 1 and O._f32(z)[0] == 8
    assert (q[0, :16] == np.arange(16)).all() and (q[0, 16:] == 0).all()
    assert (O.values(q, s, z) == x).all()


def test_quantiser_error_is_bounded_by_half_a_step():
    """|x - value| <= s/2 + what rounding s and z can add at the ends: s and z are
    each off by 2^-8 relative, so the top code's reach max - (z + 7 s) is at most
    15 * 2^-8 s + 2^-8 (|min| + 8 s) + 2^-8 |z| beyond half a step."""
    g = np.random.default_rng(0)
    x = (g.standard_normal((500, 128)) * np.exp(g.uniform(-20, 20, (500, 1)))).astype(np.float32)
    q, s, z = O.quantise(x)
    v = O.values(q, s, z)
    sf, zf = O._f32(s).astype(np.float64), O._f32(z).astype(np.float64)
    bound = sf * (0.5 + 15 / 256) + (np.abs(zf) + np.abs(x).max(1) + 8 * sf) / 256
    assert (np.abs(v - x).max(1) <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
def test_row_bytes_round_trip(d):
    g = np.random.default_rng(d)
    for r in range(8):
        q = g.integers(0, 16, d).astype(np.uint8)
        b = O.row_bytes(q, r)
        assert (O.row_codes(b, r) == q).all()
        # (word >> 4j) & 0x000F000F is the dim pair (8w + 2j, 8w + 2j + 1).
        words = b.view("<u4")
        if d == 128 and (r >> 1) & 1:
            words = np.concatenate([words[8:], words[:8]])
        for w, word in enumerate(words):
            for j in range(4):
                pair = (int(word) >> (4 * j)) & 0x000F000F
                assert (pair & 15, pair >> 16) == (q[8 * w + 2 * j], q[8 * w + 2 * j + 1])


def test_special_rows():
    x = np.zeros((6, 64), dtype=np.float32)
    x[1] = 3.5                    # constant
    x[2, 5] = np.inf
    x[3, 9] = np.nan
    x[4, :32], x[4, 32:] = 3.3e38, -3.3e38
    x[5] = 1e-40                  # subnormal
    q, s, z = O.quantise(x)
    v = O.values(q, s, z)
    assert (v[0] == 0).all() and (v[1] == 3.5).all()
    assert np.isnan(v[2]).all() and np.isnan(v[3]).all()
    assert np.isfinite(v[4]).all() and np.abs(v[4] / x[4] - 1).max() < 0.05
    assert np.abs(v[5] - x[5]).max() <= 1e-40


def test_pages_reserve_and_trim_restore_the_stack():
    table = [[7, -1, -1, -1], [-1] * 4, [3, 5, -1, -1]]
    free = [0, 1, 2, 4, 6, 99, 99, 99]
    t1, u1, f1, n1, slots, codes = O.pages_update(table, [1, 0, 2], free, 5, [10, 0, 31], [7, 20, 2], 20, 16)
    assert not codes and n1 == 1 and u1 == [2, 2, 3]
    assert t1 == [[7, 6, -1, -1], [4, 2, -1, -1], [3, 5, 1, -1]]
    assert slots[0][:7] == [122, 123, 124, 125, 126, 127, 96] and slots[0][7] == -1
    assert slots[2][:2] == [95, 16]
    t2, u2, f2, n2, _, codes = O.pages_update(t1, u1, f1, n1, [10, 0, 31], None, 0, 16)
    assert (t2, u2, f2, n2) == (table, [1, 0, 2], free, 5) and not codes


def test_logprobs_of_a_uniform_row():
    lp, ent, lse, top, ids = O.logprobs(np.zeros((1, 8)), 1.0, [[3, -1]], 2)
    assert np.allclose(lp, [[-np.log(8), 0]]) and np.allclose(ent, np.log(8)) and np.allclose(lse, np.log(8))
    assert ids.tolist() == [[0, 1]] and np.allclose(top, -np.log(8))


# ------------------------------------------------------------------ refusals
def _mem():
    buf = (ctypes.c_uint8 * 4096)()
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


def test_page_bytes(L):
    assert L.w12_kv4_page_bytes(8, 128, 64) == 8 * 64 * 136
    assert L.w12_kv4_page_bytes(1, 64, 16) == 16 * 72
    for bad in ((8, 96, 64), (8, 128, 48), (0, 128, 64), (8, 128, 256)):
        assert L.w12_kv4_page_bytes(*bad) == 0


def test_pages_refusals(L):
    buf, a = _mem()
    ok = dict(table=a, used=a, free=a, n_free=a, B=2, mp=4, P=16, n=8, start=a, add=a, T=4, slots=a)

    def call(**kw):
        v = dict(ok, **kw)
        return L.w12_pages_update(v["table"], v["used"], v["free"], v["n_free"], v["B"], v["mp"], v["P"], v["n"],
                                  v["start"], v["add"], v["T"], v["slots"], None, None)
    for name in ("table", "used", "free", "n_free", "start", "add", "slots"):
        assert call(**{name: None}) == 1, name
    assert call(T=-1) == 1
    for kw in (dict(B=0), dict(B=8193), dict(mp=0), dict(P=24), dict(n=0), dict(n=2 ** 27), dict(mp=2 ** 30)):
        assert call(**kw) == 2, kw


def test_kv4_row_refusals(L):
    buf, a = _mem()
    c = w12._KV4(a, 4, 2, 128, 64)

    def append(c=c, K=a, V=a, dt=1, n=1, slots=a):
        return L.w12_kv4_append(ctypes.byref(c), K, V, dt, n, 256, 128, 256, 128, slots, None, None)
    assert append(K=None) == 1 and append(V=None) == 1 and append(slots=None) == 1
    assert append(dt=3) == 1 and append(dt=-1) == 1 and append(n=-1) == 1
    assert append(K=a + 1) == 1                                          # not even element-aligned
    assert append(c=w12._KV4(a + 8, 4, 2, 128, 64)) == 1
    assert append(c=w12._KV4(None, 4, 2, 128, 64)) == 1
    assert append(c=w12._KV4(a, 4, 2, 96, 64)) == 2
    assert append(c=w12._KV4(a, 4, 2, 128, 20)) == 2
    assert append(c=w12._KV4(a, 2 ** 26, 2, 128, 64)) == 2               # slots would pass int32
    assert L.w12_kv4_read(ctypes.byref(c), a, 1, a + 2, a, None, None) == 1

    def commit(arr, n=1, B=1, table=a, mp=1, path=a, stride=4):
        return L.w12_kv4_commit(arr, n, B, table, mp, a, path, stride, a, None, None, None)
    one = (w12._KV4 * 1)(c)
    assert commit(one, n=0) == 1 and commit(one, B=0) == 1 and commit(one, table=None) == 1
    assert commit(one, mp=0) == 1 and commit(one, path=None) == 1 and commit(one, stride=0) == 1
    two = (w12._KV4 * 2)(c, w12._KV4(a, 4, 2, 64, 64))                   # layouts differ
    assert commit(two, n=2) == 2


def test_kv4_attention_refusals(L):
    assert L.w12_kv4_attention_ws_bytes(4, 16, 40, 8, 128, 64, 8192) > 0
    for bad in ((0, 16, 40, 8, 128, 64, 8192), (4, 0, 40, 8, 128, 64, 8192), (4, 16, 40, 7, 128, 64, 8192),
                (4, 16, 40, 8, 80, 64, 8192), (4, 16, 40, 8, 128, 63, 8192), (4, 16, 40, 8, 128, 64, 0)):
        assert L.w12_kv4_attention_ws_bytes(*bad) == 0, bad
    buf, a = _mem()
    ok = dict(q=a, s0=1 << 12, s1=512, s2=128, pool=a, table=a, mp=4, B=1, T=4, Hq=4, L=256, prefix=a, qlen=None,
              par=None, scale=0.1, o=a, ws=a, wsb=1 << 40, hd=128, P=64)

    def call(**kw):
        v = dict(ok, **kw)
        c = w12._KV4(v["pool"], 8, 2, v["hd"], v["P"])
        return L.w12_kv4_attention(v["q"], v["s0"], v["s1"], v["s2"], ctypes.byref(c), v["table"], v["mp"], v["B"],
                                   v["T"], v["Hq"], v["L"], v["prefix"], v["qlen"], v["par"], v["scale"], v["o"],
                                   v["ws"], v["wsb"], None, None)
    for name in ("q", "pool", "table", "prefix", "o"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(q=a + 2), dict(o=a + 8), dict(s1=516), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert call(**kw) == 1, kw
    for kw in (dict(L=257), dict(T=0), dict(Hq=3), dict(hd=72), dict(mp=0), dict(par=a, T=129, s0=1 << 20)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(wsb=0), dict(ws=a + 8)):
        assert call(**kw) == 3, kw


def test_logprobs_refusals(L):
    assert L.w12_logprobs_ws_bytes(16, 151936, 20) > 0
    for bad in ((0, 100, 0), (65536, 100, 0), (1, 0, 0), (1, 100, 33), (1, 100, -1), (1, 1 << 30, 0)):
        assert L.w12_logprobs_ws_bytes(*bad) == 0, bad
    buf, a = _mem()
    ok = dict(x=a, dt=0, M=2, V=100, pitch=100, scale=1.0, tok=a, n=1, k=4, lp=a, e=a, lse=a, tl=a, ti=a, ws=a, wsb=1 << 40)

    def call(**kw):
        v = dict(ok, **kw)
        return L.w12_logprobs(v["x"], v["dt"], v["M"], v["V"], v["pitch"], v["scale"], v["tok"], v["n"], v["k"], v["lp"],
                              v["e"], v["lse"], v["tl"], v["ti"], v["ws"], v["wsb"], None, None)
    for name in ("x", "tok", "lp", "e", "lse", "tl", "ti"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(dt=3), dict(x=a + 2), dict(scale=0.0), dict(n=-1), dict(scale=float("inf"))):
        assert call(**kw) == 1, kw
    for kw in (dict(pitch=99), dict(k=33), dict(M=0), dict(V=0)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(wsb=16), dict(ws=a + 4)):
        assert call(**kw) == 3, kw


def test_without_gpu_the_new_operators_are_unsupported(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    buf, a = _mem()
    c = w12._KV4(a, 4, 2, 128, 64)
    assert L.w12_pages_update(a, a, a, a, 2, 4, 16, 8, a, a, 4, a, None, None) == 8
    assert L.w12_kv4_append(ctypes.byref(c), a, a, 1, 1, 256, 128, 256, 128, a, None, None) == 8
    assert L.w12_kv4_read(ctypes.byref(c), a, 1, a, a, None, None) == 8
    assert L.w12_logprobs(a, 0, 2, 100, 100, 1.0, a, 1, 4, a, a, a, a, a, a, 1 << 40, None, None) == 8
