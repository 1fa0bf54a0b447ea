"""Norms of heads with the rotation, rotated cache appends and tree positions on the GPU. Keys are
exact: every step is one IEEE fp32 operation, and the norm's factor is the fp32 value next to the
exact one; what is rounded to 16 bits is the exact value's rounding. Queries are plain fp32: the sum of
squares passes 12 roundings (6 2^-24 of its root), the factor 2 more, the products with it and the
weight 2, the rotation's sum of two products 2 of either: 12 2^-24 of both values of a pair, so at most
24 2^-24 of the row's largest before the rotation, which is at most sqrt(2) of the largest behind it."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as KO
from oracle import layer_oracle as O
from speculative_decoding_verification_w12_gb300 import synthetic as S
from speculative_decoding_verification_w12_gb300 import w12

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _rows(n, heads, d, dtype, seed, extra=0, offset=0, scale=1.7):
    """Views [n, H, d] of one wide buffer, one behind the other."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = (torch.randn((n, sum(heads) * d + extra + offset), generator=g, device="cuda") * scale + 0.2).to(dtype)
    out, at = [], offset
    for H in heads:
        out.append(wide[:, at:at + H * d].unflatten(1, (H, d)))
        at += H * d
    return out


def _make(d, rot, pairs, norm, max_pos, seed=3):
    g = np.random.default_rng(seed)
    qw, kw = (g.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2))
    if norm == "q":
        kw = None
    elif not norm:
        qw = kw = None
    tab = O.table(max_pos, rot)
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    return w12.Rope(dev(tab), d, dev(qw), dev(kw), 1e-6, pairs), tab, qw, kw


def _same(got, want):
    """Bits of a GPU tensor and of oracle fp32 rows rounded to its type (any NaN is a NaN)."""
    want = torch.from_numpy(want).to(got.dtype).float().numpy()
    got = got.float().cpu().numpy()
    assert got.shape == want.shape
    np.testing.assert_array_equal(got, want)


def _near(got, want):
    """Queries: see the top; and the rounding to the output's type."""
    u = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}[got.dtype]
    got, want = got.float().cpu().numpy().astype(np.float64), want.astype(np.float64)
    assert got.shape == want.shape
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    off = 24 * 2.0 ** -24 * 1.4143 * np.where(fine, np.abs(want), 0).max(-1, keepdims=True)
    tol = (1 + u) * off + u * np.abs(want) + (2.0 ** -25 if u else 0)
    assert (np.abs(got - want)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,pairs,norm,out", [
    (1, 1, 1, 64, 64, False, True, BF16), (16, 40, 8, 128, 128, False, True, BF16), (33, 5, 1, 128, 64, False, True, F32),
    (7, 3, 2, 128, 32, False, "q", F16), (19, 10, 2, 64, 16, True, True, F32), (5, 12, 4, 128, 128, True, False, BF16),
    (130, 2, 1, 64, 32, False, False, F16), (3, 7, 7, 128, 112, False, True, F32), (9, 1, 1, 64, 48, True, True, BF16)])
def test_rows(n, Hq, Hkv, d, rot, pairs, norm, out, dtype):
    rope, tab, qw, kw = _make(d, rot, pairs, norm, 97)
    Q, K = _rows(n, (Hq, Hkv), d, dtype, n + d)
    pos = np.random.default_rng(n).integers(0, 97, n)
    pos[0] = 96
    pos[n // 2] = 0
    st = new_status()
    q, k = rope.run(Q, K, to_dev_i32(pos), dtype=out, status=st)
    assert status_value(st) == 0 and q.is_contiguous() and k.is_contiguous()
    _near(q, O.rope(Q.float().cpu().numpy(), qw, 1e-6, pos, tab, pairs))
    _same(k, O.rope(K.float().cpu().numpy(), kw, 1e-6, pos, tab, pairs))


@pytest.mark.parametrize("dtype,extra,offset", [(F32, 3, 1), (BF16, 5, 0), (F16, 8, 8), (BF16, 1, 7), (F32, 4, 4)])
def test_strided_and_unaligned_views(dtype, extra, offset):
    rope, tab, qw, kw = _make(128, 128, False, True, 40)
    Q, K = _rows(11, (3, 2), 128, dtype, 5, extra, offset)
    pos = np.arange(11)
    q, k = rope.run(Q, K, to_dev_i32(pos), dtype=F32)
    _near(q, O.rope(Q.float().cpu().numpy(), qw, 1e-6, pos, tab))
    _same(k, O.rope(K.float().cpu().numpy(), kw, 1e-6, pos, tab))


def test_transposed_and_broadcast_rows():
    rope, tab, qw, kw = _make(64, 64, False, True, 40)
    Q = _rows(6, (4,), 64, F32, 1)[0].permute(1, 0, 2)      # heads become tokens
    K = _rows(1, (2,), 64, F32, 2)[0].expand(4, 2, 64)      # one row for all tokens
    pos = np.array([3, 39, 0, 11])
    q, k = rope.run(Q, K, to_dev_i32(pos), dtype=F32)
    _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, pos, tab))
    _same(k, O.rope(K.cpu().numpy(), kw, 1e-6, pos, tab))


def test_queries_or_keys_alone_and_given_outputs():
    rope, tab, qw, kw = _make(64, 32, True, True, 40)
    Q, K = _rows(6, (4, 2), 64, BF16, 1)
    pos = to_dev_i32(np.arange(6))
    both = rope.run(Q, K, pos)
    q, none = rope.run(Q, None, pos)
    assert none is None and torch.equal(q, both[0])
    none, k = rope.run(None, K, pos)
    assert none is None and torch.equal(k, both[1])
    out = tuple(torch.full_like(x, 7) for x in both)
    assert rope.run(Q, K, pos, out=out)[0].data_ptr() == out[0].data_ptr()
    assert torch.equal(out[0], both[0]) and torch.equal(out[1], both[1])
    empty = rope.run(Q[:0], K[:0], pos[:0])
    assert empty[0].shape == (0, 4, 64) and empty[1].shape == (0, 2, 64)


def test_positions_without_a_token_and_outside_the_table():
    rope, tab, qw, kw = _make(128, 128, False, True, 40)
    Q, K = _rows(5, (3, 1), 128, F32, 1)
    pos = np.array([0, -1, 39, -1, 5])
    st = new_status()
    q, _ = rope.run(Q, K, to_dev_i32(pos), dtype=F32, status=st)
    assert status_value(st) == 0
    _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, pos, tab))
    for bad in (40, -2, 2 ** 31 - 1, -2 ** 31):
        st = new_status()
        q, k = rope.run(Q, K, to_dev_i32(np.array([0, bad, 39, -1, 5])), dtype=F32, status=st)
        assert status_value(st) == 1
        _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, pos, tab))


def test_rows_of_any_size():
    """Squares past the fp32 range, below it, and constant rows."""
    rope, tab, qw, kw = _make(128, 128, False, True, 40)
    Q, K = _rows(9, (2, 1), 128, F32, 1)
    size = torch.tensor([1e-38, 1e-20, 1e-3, 1.0, 1e10, 3e18, 1e25, 1e38, 0.0], device="cuda")[:, None, None]
    Q, K = Q.contiguous() * size, K.contiguous() * size
    Q[3] = 2.0
    pos = np.arange(9)
    q, k = rope.run(Q, K, to_dev_i32(pos), dtype=F32)
    _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, pos, tab))
    q, want = k, O.rope(K.cpu().numpy(), kw, 1e-6, pos, tab)
    _same(q[:6], want[:6])
    # (Past 2^63 the factor is rounded with two exponents: 2^-23 of the value. Some of the rows near
    # 1e38 have gone to infinity: the factor is 0, and infinity times it NaN.)
    got = q[6:].cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want[6:]))
    fine = ~np.isnan(got)
    assert np.abs(got - want[6:])[fine].max() <= 2.0 ** -22 * np.abs(want[6:][fine]).max()


def test_rows_near_the_end_of_the_range():
    rope, tab, qw, kw = _make(64, 64, False, True, 40)
    Q = _rows(9, (2,), 64, F32, 1)[0].contiguous() * 2e37
    assert torch.isfinite(Q).all()
    q, k = rope.run(Q, Q, to_dev_i32(np.arange(9)), dtype=F32)
    want = O.rope(Q.cpu().numpy(), kw, 1e-6, np.arange(9), tab)
    assert np.abs(k.cpu().numpy() - want).max() <= 2.0 ** -22 * np.abs(want).max() and np.abs(want).max() > 1
    _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, np.arange(9), tab))


def test_many_keys():
    """The factor is the nearest fp32 value; one that two are almost as near to may go either way (the
    sums know it to about 2^-16 of their distance), which moves a value by two roundings."""
    rope, tab, qw, kw = _make(128, 128, False, True, 500)
    for dtype in (F32, BF16, F16):
        K = _rows(500, (8,), 128, dtype, 11)[0]
        pos = np.arange(500)
        k = rope.run(None, K, to_dev_i32(pos), dtype=F32)[1].cpu().numpy()
        want = O.rope(K.float().cpu().numpy(), kw, 1e-6, pos, tab)
        other = (k != want).any(-1)
        assert other.sum() <= 2
        assert np.abs(k - want).max() <= 2.0 ** -22 * np.abs(want).max()


def test_values_that_are_not_finite_stay_in_their_row():
    rope, tab, qw, kw = _make(64, 64, False, True, 40)
    Q, K = _rows(8, (4, 2), 64, F32, 1)
    clean = rope.run(Q, K, to_dev_i32(np.arange(8)), dtype=F32)[0]
    Q = Q.contiguous()
    Q[1, 2, 5], Q[3, 0, 63], Q[6, 1, 0] = float("nan"), float("inf"), float("-inf")
    q, k = rope.run(Q, Q, to_dev_i32(np.arange(8)), dtype=F32)
    keep = torch.ones((8, 4), dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[3, 0] = keep[6, 1] = False
    assert torch.equal(q[keep], clean[keep])
    _near(q, O.rope(Q.cpu().numpy(), qw, 1e-6, np.arange(8), tab))
    _same(k, O.rope(Q.cpu().numpy(), kw, 1e-6, np.arange(8), tab))


def _pool(n_pages, Hkv, d, P):
    c = w12.KV4Cache.create(n_pages, Hkv, d, P)
    c.pool.fill_(0xA5)
    return c


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,pairs,norm,P", [
    (1, 0, 1, 128, 128, False, True, 16), (37, 15, 3, 128, 128, False, True, 64), (16, 0, 8, 64, 32, False, True, 32),
    (5, 10, 2, 128, 32, True, False, 128), (70, 1, 1, 64, 64, True, True, 16), (9, 4, 4, 128, 64, False, False, 32)])
def test_append_bytes(n, Hq, Hkv, d, rot, pairs, norm, P, dtype):
    rope, tab, qw, kw = _make(d, rot, pairs, norm, 97)
    rows = _rows(n, (Hq, Hkv, Hkv) if Hq else (Hkv, Hkv), d, dtype, n + d)
    Q, (K, V) = (rows[0], rows[1:]) if Hq else (None, rows)
    g = np.random.default_rng(n)
    slots = g.permutation(n * 3)[:n].astype(int).tolist()
    pos = g.integers(0, 97, n)
    if n > 1:
        slots[n // 2] = -1                        # no slot
        pos[n // 3] = -1                          # no token
    c = _pool(max(slots) // P + 2, Hkv, d, P)
    before = c.pool.cpu().numpy()
    st = new_status()
    q = c.append_rope(K, V, to_dev_i32(slots), rope, to_dev_i32(pos), Q=Q, status=st)
    assert status_value(st) == 0
    kept = [-1 if p < 0 else s for s, p in zip(slots, pos)]
    want = KO.append(before, O.rope(K.float().cpu().numpy(), kw, 1e-6, pos, tab, pairs), V.float().cpu().numpy(), kept, d)
    assert (c.pool.cpu().numpy() == want).all()
    if Hq:
        assert q.dtype is BF16
        _near(q, O.rope(Q.float().cpu().numpy(), qw, 1e-6, pos, tab, pairs))
    else:
        assert q is None
    # The same in two calls: rotated to fp32, then appended.
    two = _pool(c.n_pages, Hkv, d, P)
    two.append(rope.run(None, K, to_dev_i32(pos), dtype=F32)[1], V.float(), to_dev_i32(kept))
    assert torch.equal(two.pool, c.pool)


def test_append_refuses_slots_and_positions_out_of_range():
    rope, *_ = _make(64, 64, False, True, 40)
    K, V = _rows(4, (2, 2), 64, F32, 1)
    for slots, pos in (([0, 1, 64, 2], [0, 1, 2, 3]), ([0, 1, -7, 2], [0, 1, 2, 3]), ([0, 1, 3, 2], [0, 1, 40, 3]), ([0, 1, 3, 2], [0, 1, -2, 3])):
        c = _pool(4, 2, 64, 16)
        st = new_status()
        c.append_rope(K, V, to_dev_i32(slots), rope, to_dev_i32(pos), status=st)
        assert status_value(st) == 1
        ref = _pool(4, 2, 64, 16)
        ref.append_rope(K, V, to_dev_i32([0, 1, -1, 2]), rope, to_dev_i32([0, 1, 2, 3]))
        assert torch.equal(c.pool, ref.pool)


def test_append_rows_that_are_not_finite():
    rope, tab, qw, kw = _make(128, 128, False, True, 40)
    K, V = (x.contiguous() for x in _rows(3, (2, 2), 128, F32, 1))
    K[0, 1, 7], V[2, 0, 100] = float("nan"), float("inf")
    c = _pool(1, 2, 128, 16)
    before = c.pool.cpu().numpy()
    c.append_rope(K, V, to_dev_i32([3, 4, 5]), rope, to_dev_i32([0, 1, 2]))
    want = KO.append(before, O.rope(K.cpu().numpy(), kw, 1e-6, [0, 1, 2], tab), V.cpu().numpy(), [3, 4, 5], 128)
    assert (c.pool.cpu().numpy() == want).all()


@pytest.mark.parametrize("B,T", [(1, 1), (3, 2), (5, 16), (2, 64), (2, 129), (3, 256)])
def test_tree_positions(B, T):
    g = np.random.default_rng(T)
    trees = np.stack([S.random_tree(T, max_depth=min(12, T), g=g) if b % 2 else np.arange(-1, T - 1) for b in range(B)])
    prefix = g.integers(0, 10000, B)
    n = g.integers(0, T + 1, B)
    n[0] = T
    for q_len in (None, n):
        st = new_status()
        ql = None if q_len is None else to_dev_i32(q_len)
        got = w12.tree_positions(to_dev_i32(prefix), to_dev_i32(trees), q_len=ql, status=st)
        assert status_value(st) == 0
        assert (got.cpu().numpy() == O.tree_positions(prefix, trees, q_len, T)).all()
        flat = w12.tree_positions(to_dev_i32(prefix), T=T, q_len=ql)
        assert (flat.cpu().numpy() == O.tree_positions(prefix, None, q_len, T)).all()


def test_positions_of_a_long_chunk_and_at_the_end_of_the_range():
    got = w12.tree_positions(to_dev_i32([7, 2 ** 31 - 1000]), T=1000)
    assert (got[0].cpu().numpy() == np.arange(7, 1007)).all() and int(got[1, -1]) == 2 ** 31 - 1
    st = new_status()
    got = w12.tree_positions(to_dev_i32([7, 2 ** 31 - 999]), T=1000, status=st)
    assert status_value(st) == 1 and (got[1] == -1).all() and int(got[0, 999]) == 1006


@pytest.mark.parametrize("tree,q_len,code", [([0, 0, 0], 3, 4), ([-1, 1, 0], 3, 4), ([-1, 0, -1], 3, 4), ([-1, 0, 5], 3, 4),
                                             ([-1, 0, 0], 4, 1), ([-1, 0, 0], -1, 1)])
def test_malformed_trees_and_lengths(tree, q_len, code):
    st = new_status()
    got = w12.tree_positions(to_dev_i32([5, 6]), to_dev_i32(np.array([tree, [-1, 0, 1]])), q_len=to_dev_i32([q_len, 3]), status=st)
    assert status_value(st) == code and got.tolist() == [[-1] * 3, [6, 7, 8]]
    # What is wrong past the request's nodes is not looked at.
    st = new_status()
    got = w12.tree_positions(to_dev_i32([5]), to_dev_i32(np.array([[-1, 0, 9]])), q_len=to_dev_i32([2]), status=st)
    assert status_value(st) == 0 and got.tolist() == [[5, 6, -1]]


def test_captured_and_replayed_on_another_stream():
    rope, tab, qw, kw = _make(128, 128, False, True, 64)
    Q, K, V = _rows(12, (5, 1, 1), 128, F32, 1)
    c = _pool(2, 1, 128, 16)
    prefix, parents, slots = to_dev_i32([3]), to_dev_i32(np.arange(-1, 11)[None]), to_dev_i32(np.arange(12))
    out = torch.empty((12, 5, 128), dtype=BF16, device="cuda")

    def step():
        c.append_rope(K, V, slots, rope, w12.tree_positions(prefix, parents)[0], Q=Q, out=out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    prefix.fill_(30)
    Q.mul_(2)
    c.pool.fill_(0xA5)
    g.replay()
    torch.cuda.synchronize()
    pos = np.arange(30, 42)
    _near(out, O.rope(Q.cpu().numpy(), qw, 1e-6, pos, tab))
    want = KO.append(np.full(c.pool.shape, 0xA5, dtype=np.uint8), O.rope(K.cpu().numpy(), kw, 1e-6, pos, tab), V.cpu().numpy(), list(range(12)), 128)
    assert (c.pool.cpu().numpy() == want).all()
    side = torch.cuda.Stream()
    q, _ = rope.run(Q, K, to_dev_i32(pos), stream=side)
    side.synchronize()
    assert torch.equal(q, out)


@pytest.mark.parametrize("d", [64, 128])
def test_the_factor_of_the_largest_rows(d):
    """Values of [2^127, 2^128): the row times 2^-76 (exact), and the fp32 value next to its factor.
    (One row of these may be a tie of two, as above.)"""
    rope, tab, qw, kw = _make(d, d, False, True, 4)
    g = torch.Generator(device="cuda").manual_seed(d)
    K = (torch.rand((200, 3, d), generator=g, device="cuda") * 0.99 + 1.0) * 2.0 ** 127
    K = torch.where(torch.rand(K.shape, generator=g, device="cuda") < 0.5, -K, K)
    assert torch.isfinite(K).all()
    k = rope.run(None, K, to_dev_i32(np.zeros(200)), dtype=F32)[1].cpu().numpy()   # (a turn by nothing)
    x = K.cpu().numpy() * np.float32(2.0 ** -76)
    f = (1 / np.sqrt(np.square(x.astype(np.float64)).mean(-1, keepdims=True))).astype(np.float32)
    want = (x * f) * kw
    assert (k != want).any(-1).sum() <= 1
    assert np.abs(k - want).max() <= 2.0 ** -22 * np.abs(want).max()


def test_rows_and_slots_past_32_bits():
    """Rows 2^23 values apart, 600 of them, and a pool of more than 2^32 bytes."""
    n, apart = 600, 2 ** 23
    rope = _make(128, 128, False, True, n)[0]
    base = torch.empty(n * apart, dtype=BF16, device="cuda")
    Q, K, V = (base.as_strided((n, h, 128), (apart, 128, 1), at) for h, at in ((3, 0), (2, 384), (2, 640)))
    g = torch.Generator(device="cuda").manual_seed(2)
    for x in (Q, K, V):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    pos, st = to_dev_i32(np.arange(n)), new_status()
    for got, want in zip(rope.run(Q, K, pos, status=st), rope.run(Q.contiguous(), K.contiguous(), pos)):
        assert torch.equal(got, want)
    P, pages = 64, 260_000
    big, small = _pool(pages, 2, 128, P), _pool(n // P + 1, 2, 128, P)
    assert big.pool.numel() > 2 ** 32
    slots = to_dev_i32(np.arange(n) + (pages - n // P - 1) * P)
    q = big.append_rope(K, V, slots, rope, pos, Q=Q, status=st)
    assert torch.equal(q, small.append_rope(K.contiguous(), V.contiguous(), pos, rope, pos, Q=Q.contiguous()))
    for got, want in zip(big.read(slots), small.read(pos)):
        assert torch.equal(got, want)
    assert status_value(st) == 0


# Rows enough for groups of heads: at least 608 blocks of 128 / (d / 16) of them.
MANY = [(3400, 5, 1, 128, 128, False, True), (5000, 10, 2, 64, 64, False, True), (3400, 6, 3, 128, 64, False, False), (2500, 7, 4, 128, 128, True, True),
        (5000, 9, 2, 64, 32, True, "q")]


def _same_or_tie(got, x, w, pos, tab, pairs):
    """As _same, among so many rows that a factor may lie in the middle of two fp32 numbers: 128 rests of
    squares of up to 2^-17 of the whole are summed in 12 fp32 additions, off by up to 12 2^-24 2^-10 of
    it, the factor by half of that, which is less than 2^-7 of the distance of two. There it is either."""
    dtype = got.dtype
    want = torch.from_numpy(O.rope(x, w, 1e-6, pos, tab, pairs)).to(dtype).float().numpy()
    got = got.float().cpu().numpy()
    n, h = np.nonzero((got != want).any(-1))
    if len(n):
        assert w is not None and len(n) <= 3
        row = x[n, h][:, None]
        r = 1 / np.sqrt(np.square(row.astype(np.float64)).mean(-1, keepdims=True) + np.float64(np.float32(1e-6)))
        near = r.astype(np.float32)
        other = np.nextafter(near, np.where(r > near, np.float32(np.inf), np.float32(0)))
        assert (np.abs(r - (near.astype(np.float64) + other) / 2) <= 2.0 ** -7 * np.abs(other - near)).all()
        want = torch.from_numpy(O.rope((row * other) * w, None, 0, pos[n], tab, pairs)).to(dtype).float().numpy()
        np.testing.assert_array_equal(got[n, h][:, None], want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,pairs,norm", MANY)
def test_many_rows_give_what_few_give(n, Hq, Hkv, d, rot, pairs, norm, dtype):
    rope, tab, qw, kw = _make(d, rot, pairs, norm, 97)
    g = np.random.default_rng(n)
    pos = g.integers(-1, 97, n)
    dev = to_dev_i32(pos)
    for offset, out in ((0, BF16), (0, F32), (3, F16)):    # (an odd offset: rows read one value at a time)
        Q, K = _rows(n, (Hq, Hkv), d, dtype, n + d, offset=offset)
        st = new_status()
        got = rope.run(Q, K, dev, dtype=out, status=st)
        few = [rope.run(Q[i:i + 90], K[i:i + 90], dev[i:i + 90], dtype=out) for i in range(0, n, 90)]
        for a, b in zip(got, zip(*few)):
            assert torch.equal(a, torch.cat(b))
        assert status_value(st) == 0
        _near(got[0], O.rope(Q.float().cpu().numpy(), qw, 1e-6, pos, tab, pairs))
        _same_or_tie(got[1], K.float().cpu().numpy(), kw, pos, tab, pairs)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,pairs,norm", MANY)
def test_many_appended_rows_give_what_few_give(n, Hq, Hkv, d, rot, pairs, norm, dtype):
    rope = _make(d, rot, pairs, norm, 97)[0]
    g = np.random.default_rng(n)
    Q, K, V = _rows(n, (Hq, Hkv, Hkv), d, dtype, n + d)
    K = torch.where(torch.rand((n, 1, 1), device="cuda") < 0.1, K * 1000, K)     # (codes that need their clamp, some rows)
    slots, pos = g.permutation(n + 100)[:n], g.integers(-1, 97, n)
    slots[g.random(n) < 0.05] = -1
    slots, pos, st = to_dev_i32(slots), to_dev_i32(pos), new_status()
    whole, parts, two = (_pool((n + 100) // 64 + 1, Hkv, d, 64) for _ in range(3))
    q = whole.append_rope(K, V, slots, rope, pos, Q=Q, status=st)
    few = [parts.append_rope(K[i:i + 90], V[i:i + 90], slots[i:i + 90], rope, pos[i:i + 90], Q=Q[i:i + 90]) for i in range(0, n, 90)]
    assert status_value(st) == 0
    assert torch.equal(q, torch.cat(few)) and torch.equal(whole.pool, parts.pool)
    two.append(rope.run(None, K, pos, dtype=F32)[1], V.float(), torch.where(pos < 0, -1, slots))
    assert torch.equal(two.pool, whole.pool)
