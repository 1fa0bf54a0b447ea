"""GPU attention over the paged 4-bit cache against the float64 oracle.

The cache is filled by the library's append (its bytes are tested exactly
elsewhere); the oracle works on the values the codes stand for.

Tolerances, from the roundings the operator may make (bf16: 2^-8 relative
each): values of the cache rounded to bf16 as operands (K: the scores of a row
move by at most eps = 2^-8 scale max_j |q|.|K_j|, its weights by a factor within
e^(2 eps)), the weights rounded to bf16, V rounded to bf16, the output rounded to
bf16. With A = sum_j p_j |V_j|, |O| <= A:
    |error| <= A (e^(2 eps) - 1 + 3 * 2^-8 + 2^-12)
(2^-12 covers the fp32 sums and the exponentials). Over a whole output those
roundings are independent: each is at most 2^-8 relative, 2^-8 / sqrt(3) in the
root mean square, so four of them stay below 2^-7 of the norm.
"""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as O
from speculative_decoding_verification_w12_gb300 import synthetic as S

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")

U = 2.0 ** -8


class Case:
    """A cache filled for requests of the given lengths, and the oracle's view of it."""

    def __init__(self, prefix, new, T, Hq, Hkv, d, P, seed=0, std=1.0, grow=None, extra_pages=2, high=False):
        g = np.random.default_rng(seed)
        self.prefix, self.new, self.T, self.Hq, self.Hkv, self.d, self.P = list(prefix), list(new), T, Hq, Hkv, d, P
        B = self.B = len(prefix)
        lens = [a + n for a, n in zip(prefix, new)]
        need = [-(-L // P) for L in lens]
        ids = g.permutation(sum(need) + extra_pages)
        if high:                               # the requests hold the pool's last pages
            ids = np.sort(ids)[::-1]
        width = max(max(need), 1) + 8
        self.table = np.full((B, width), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.K, self.V, slots = [], [], []
        rows = []
        for b, L in enumerate(lens):
            kv = (g.standard_normal((2, L, Hkv, d)) * std).astype(np.float32)
            if grow:
                kv[0] *= np.linspace(grow[0], grow[1], max(L, 1), dtype=np.float32)[:L, None, None]
            rows.append(kv)
            self.K.append(O.values(*O.quantise(kv[0])))
            self.V.append(O.values(*O.quantise(kv[1])))
            pos = np.arange(L)
            slots.append(self.table[b, pos // P] * P + pos % P)
        # Every byte that no request's row covers is 0xFF: parameters that are NaN.
        self.cache = w12.KV4Cache(torch.full((len(ids), Hkv, P * (d + 8)), 255, dtype=torch.uint8, device="cuda"), P, d)
        kv = torch.from_numpy(np.concatenate(rows, 1)).cuda()
        self.cache.append(kv[0], kv[1], to_dev_i32(np.concatenate(slots)))
        self.slots = slots
        self.Q = torch.from_numpy(g.standard_normal((B, T, Hq, d)).astype(np.float32)).cuda().bfloat16()
        self.parents = None

    def trees(self, seed=1, bad=None):
        g = np.random.default_rng(seed)
        self.parents = np.stack([S.random_tree(self.T, max_depth=min(12, self.T - 1), g=g) for _ in range(self.B)])
        return self

    def run(self, scale=None, Q=None, max_len=None, status=None, q_len=True, att=None, **kw):
        L = max(a + n for a, n in zip(self.prefix, self.new)) if max_len is None else max_len
        att = att or w12.KV4Attention(self.B, self.T, self.Hq, self.Hkv, self.d, self.P, max(L, 1))
        return att.run(self.Q if Q is None else Q, self.cache, to_dev_i32(self.table), to_dev_i32(self.prefix),
                       parents=None if self.parents is None else to_dev_i32(self.parents),
                       q_len=to_dev_i32(self.new) if q_len else None, scale=scale, status=status, **kw)

    def check(self, out, scale=None, heads=None):
        scale = self.d ** -0.5 if scale is None else scale
        out = out.float().cpu().numpy().astype(np.float64)
        Q = self.Q.float().cpu().numpy().astype(np.float64)
        err2 = ref2 = 0.0
        for b in range(self.B):
            n = self.new[b]
            assert (out[b, n:] == 0).all(), f"rows past the request's tokens, b={b}"
            if n == 0:
                continue
            see = O.visible(self.prefix[b], n, None if self.parents is None else self.parents[b])
            groups = range(self.Hkv) if heads is None else heads
            G = self.Hq // self.Hkv
            for h in groups:
                hs = slice(h * G, (h + 1) * G)
                ref, A, E = O.attention(Q[b, :n, hs], self.K[b][:, h:h + 1], self.V[b][:, h:h + 1], see, scale)
                err = out[b, :n, hs] - ref
                assert np.isfinite(out[b, :n, hs]).all(), f"b={b} h={h}"
                bound = A * (np.expm1(2 * U * E)[..., None] + 3 * U + 2.0 ** -12) + 1e-30
                worst = np.unravel_index(np.argmax(np.abs(err) - bound), err.shape)
                assert (np.abs(err) <= bound).all(), f"b={b} h={h} {worst}: {err[worst]} above {bound[worst]}"
                err2 += (err ** 2).sum()
                ref2 += (ref ** 2).sum()
        rel = (err2 / max(ref2, 1e-300)) ** 0.5
        assert rel <= 2.0 ** -7, f"relative error {rel}"
        return rel


LAYOUTS = [(40, 8, 128, 64), (8, 8, 64, 16), (16, 1, 128, 32), (12, 4, 64, 128), (7, 7, 128, 128), (10, 2, 128, 16)]


@pytest.mark.parametrize("Hq,Hkv,d,P", LAYOUTS)
@pytest.mark.parametrize("prefix", [[0], [1, 0, 15], [16, 17, 127, 128, 129], [700, 3, 1023]])
def test_single_tokens(Hq, Hkv, d, P, prefix):
    c = Case(prefix, [1] * len(prefix), 1, Hq, Hkv, d, P, seed=len(prefix) + Hq)
    st = new_status()
    c.check(c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("Hq,Hkv,d,P", LAYOUTS)
@pytest.mark.parametrize("T,prefix,new", [(2, [5, 130], [2, 1]), (16, [0, 300, 112], [16, 16, 3]), (7, [1, 64, 513], [0, 7, 5]),
                                          (33, [127, 40], [33, 20])])
def test_drafted_blocks(Hq, Hkv, d, P, T, prefix, new):
    c = Case(prefix, new, T, Hq, Hkv, d, P, seed=T + Hq)
    st = new_status()
    c.check(c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("Hq,Hkv,d,P", [(40, 8, 128, 64), (10, 2, 64, 16), (2, 2, 128, 128), (16, 1, 64, 32)])
@pytest.mark.parametrize("T,prefix,new", [(16, [0, 301], [16, 9]), (64, [129, 777], [64, 40]), (128, [60], [128]), (3, [10, 128], [3, 2]), (1, [37], [1])])
def test_draft_trees(Hq, Hkv, d, P, T, prefix, new):
    c = Case(prefix, new, T, Hq, Hkv, d, P, seed=T).trees(T)
    st = new_status()
    c.check(c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("Hq,Hkv,d,P,T,prefix,new", [(4, 2, 64, 32, 500, [0, 100], [500, 333]), (5, 1, 128, 64, 257, [1000], [257]),
                                                     (3, 3, 128, 16, 1100, [0], [1100]), (16, 2, 64, 128, 130, [31, 0, 9], [130, 0, 129])])
def test_prompt_chunks(Hq, Hkv, d, P, T, prefix, new):
    c = Case(prefix, new, T, Hq, Hkv, d, P, seed=T)
    st = new_status()
    c.check(c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("T,tree", [(1, False), (16, False), (64, True)])
def test_long_cache_split_over_the_gpu(T, tree):
    """One long and one short request: the keys of a head are split and joined."""
    c = Case([20000, 17], [T, T], T, 10, 2, 128, 64, seed=T)
    if tree:
        c.trees()
    st = new_status()
    c.check(c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("T", [1, 16, 150])
def test_many_requests_of_uneven_length(T):
    g = np.random.default_rng(T)
    B = 40
    prefix = g.integers(0, 900, B)
    prefix[:3] = [0, 899, 128]
    new = g.integers(0, T + 1, B)
    new[3] = 0
    c = Case(prefix.tolist(), new.tolist(), T, 8, 4, 64, 32, seed=T)
    st = new_status()
    c.check(c.run(status=st, max_len=1100))
    assert status_value(st) == 0


@pytest.mark.parametrize("T", [1, 16, 40])
def test_peaked_and_growing_scores(T):
    """A large scale, and keys that grow along the sequence: the running maximum keeps moving."""
    c = Case([1500], [T], T, 5, 1, 128, 64, seed=2, grow=(0.2, 1.0))
    c.check(c.run(scale=0.4), scale=0.4)
    c = Case([1500], [T], T, 5, 1, 128, 64, seed=2, grow=(1.0, 0.1))
    c.check(c.run(scale=0.4), scale=0.4)


@pytest.mark.parametrize("T", [1, 16])
def test_large_centres(T):
    """Rows far from zero (centre 40, spread 1): the centre does not eat the codes."""
    c = Case([300], [T], T, 8, 2, 128, 64, seed=6)
    g = np.random.default_rng(7)
    L = 300 + T
    kv = (g.standard_normal((2, L, 2, 128)) + 40).astype(np.float32)
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[0]))
    c.K, c.V = [O.values(*O.quantise(kv[0]))], [O.values(*O.quantise(kv[1]))]
    c.check(c.run(scale=0.01), scale=0.01)


@pytest.mark.parametrize("T,Hq,Hkv", [(16, 5, 1), (1, 4, 4), (4, 4, 1)])
def test_values_that_are_not_finite_stay_in_masked_places(T, Hq, Hkv):
    """Tree nodes with NaN keys or values: only the rows that see them are NaN."""
    c = Case([200] * 2, [T, T], T, Hq, Hkv, 128, 64, seed=8)
    c.trees(3)
    if T > 1:
        # Node T - 1 is nobody's ancestor; node 1's subtree sees node 1.
        x = torch.full((2, Hkv, 128), float("nan"), device="cuda")
        y = torch.ones((2, Hkv, 128), device="cuda")
        c.cache.append(x, y, to_dev_i32([c.slots[0][200 + T - 1], c.slots[1][200 + 1]]))
        out = c.run().float()
        anc = [O.visible(200, T, c.parents[b]) for b in range(2)]
        for b, node in ((0, T - 1), (1, 1)):
            for t in range(T):
                assert torch.isnan(out[b, t]).all() == bool(anc[b][t, 200 + node]), (b, t)
                assert torch.isnan(out[b, t]).any() == bool(anc[b][t, 200 + node]), (b, t)
        c.cache.append(y, x, to_dev_i32([c.slots[0][200 + T - 1], c.slots[1][200 + 1]]))
        out = c.run().float()
        for b, node in ((0, T - 1), (1, 1)):
            for t in range(T):
                assert torch.isnan(out[b, t]).all() == bool(anc[b][t, 200 + node]), (b, t)
                assert torch.isnan(out[b, t]).any() == bool(anc[b][t, 200 + node]), (b, t)
    else:
        c.check(c.run())


@pytest.mark.parametrize("T", [1, 3, 16, 200])
def test_query_views_and_given_output(T):
    """Q as a slice of a wider product, heads and tokens in another order."""
    c = Case([130, 9], [T, T], T, 6, 2, 64, 32, seed=9)
    wide = torch.zeros((2, T, 8, 64 + 8), dtype=torch.bfloat16, device="cuda")
    view = wide[:, :, 1:7, 8:]
    view.copy_(c.Q)
    out = torch.full((2, T, 6, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert c.run(Q=view, out=out) is out
    c.check(out)
    other = torch.empty((6, 2, T, 64), dtype=torch.bfloat16, device="cuda").permute(1, 2, 0, 3)
    other.copy_(c.Q)
    c.check(c.run(Q=other))


@pytest.mark.parametrize("T", [1, 16, 64])
def test_workspace_reused_streams_and_graph(T):
    c = Case([3000, 50], [T, T], T, 5, 1, 128, 64, seed=10)
    att = w12.KV4Attention(2, T, 5, 1, 128, 64, 3000 + T)
    first = c.run(att=att)
    c.check(first)
    for _ in range(3):
        assert (c.run(att=att) == first).all()                       # the same result, bit for bit
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(att=att, stream=s)
    s.synchronize()
    assert (out == first).all()
    args = (c.Q, c.cache, to_dev_i32(c.table), to_dev_i32(c.prefix))
    res = torch.empty_like(first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att.run(*args, out=res)
    for _ in range(2):
        res.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert (res == first).all()


@pytest.mark.parametrize("T", [1, 16, 200])
def test_default_new_lengths(T):
    c = Case([70, 0], [T, T], T, 4, 2, 64, 16, seed=11)
    c.check(c.run(q_len=False))


def test_bad_lengths_trees_and_pages_are_flagged():
    c = Case([40], [8], 8, 4, 2, 64, 16, seed=12)
    att = lambda: w12.KV4Attention(1, 8, 4, 2, 64, 16, 48)  # noqa: E731

    def code(prefix=(40,), new=(8,), table=None, parents=None):
        st = new_status()
        att().run(c.Q, c.cache, to_dev_i32(c.table if table is None else table), to_dev_i32(prefix),
                  parents=None if parents is None else to_dev_i32(parents), q_len=to_dev_i32(new), status=st)
        return status_value(st)
    assert code() == 0
    assert code(prefix=(41,)) == 1 and code(prefix=(-1,)) == 1 and code(new=(9,)) == 1 and code(new=(-1,)) == 1
    bad = c.table.copy()
    bad[0, 1] = c.cache.n_pages
    assert code(table=bad) == 1
    bad[0, 1] = -1
    assert code(table=bad) == 1
    assert code(parents=[[-1, 0, 1, 5, 2, 3, 4, 5]]) == 4
    assert code(parents=[[0, 0, 1, 2, 2, 3, 4, 5]]) == 4


def test_binding_refusals():
    c = Case([40], [8], 8, 4, 2, 64, 16, seed=12)
    att = w12.KV4Attention(1, 8, 4, 2, 64, 16, 48)
    tab, pre = to_dev_i32(c.table), to_dev_i32(c.prefix)
    for Q in (c.Q.float(), c.Q[:, :7], c.Q.cpu(), c.Q.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            att.run(Q, c.cache, tab, pre)
    with pytest.raises(ValueError):
        att.run(c.Q, c.cache, tab.long(), pre)
    with pytest.raises(ValueError):
        att.run(c.Q, c.cache, tab, to_dev_i32([1, 2]))
    with pytest.raises(ValueError):
        att.run(c.Q, w12.KV4Cache.create(2, 2, 64, 32), tab, pre)
    with pytest.raises(ValueError):
        att.run(c.Q, c.cache, tab, pre, parents=to_dev_i32([[-1, 0]]))
    with pytest.raises(w12.W12Error) as e:
        att.run(c.Q, c.cache, tab, pre, scale=0.0)
    assert e.value.code == 1
    with pytest.raises(w12.W12Error) as e:
        w12.KV4Attention(1, 8, 4, 2, 64, 16, 200).run(c.Q, c.cache, tab, pre)      # max_kv_len past the table
    assert e.value.code == 2
    with pytest.raises(w12.W12Error):
        w12.KV4Attention(1, 8, 4, 3, 64, 16, 48)


@pytest.mark.parametrize("T", [1, 16])
def test_pages_past_4_gigabytes(T):
    """Byte offsets of pages pass 32 bits."""
    c = Case([300, 500], [T, T], T, 40, 8, 128, 128, seed=13, extra_pages=(9 << 29) // (8 * 128 * 136),
             high=True)
    assert c.cache.pool.numel() > 1 << 32 and int(c.table[c.table >= 0].min()) * 8 * 128 * 136 > 1 << 32
    c.check(c.run(), heads=(0, 7))


@pytest.mark.parametrize("scale", [1e-20, 1e20])
@pytest.mark.parametrize("T", [1, 16])
def test_queries_far_from_one(T, scale):
    """Queries of 1e20 with a small scale, and the reverse: rows keep powers of two of their own."""
    c = Case([200], [T], T, 8, 2, 64, 32, seed=14)
    c.Q = (c.Q.float() * scale).bfloat16()
    c.check(c.run(scale=0.125 / scale), scale=float(np.float32(0.125 / scale)))


@pytest.mark.parametrize("T", [1, 16])
def test_values_of_very_different_size(T):
    """Keys whose value rows are 1e-12, 1 and 1e12 large, in runs and alternating."""
    c = Case([400], [T], T, 8, 2, 128, 64, seed=15)
    g = np.random.default_rng(16)
    L = 400 + T
    size = np.ones(L, dtype=np.float32)
    size[:128], size[128:260], size[300:] = 1e-12, 1e12, 1e-12
    size[301::2] = 1.0
    kv = g.standard_normal((2, L, 2, 128)).astype(np.float32)
    kv[1] *= size[:, None, None]
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[0]))
    c.K, c.V = [O.values(*O.quantise(kv[0]))], [O.values(*O.quantise(kv[1]))]
    c.check(c.run())
    # Rows that see the tiny values alone keep them: a tree whose prefix is tiny throughout.
    kv[1] = g.standard_normal(kv[1].shape).astype(np.float32) * np.float32(1e-12)
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[0]))
    c.V = [O.values(*O.quantise(kv[1]))]
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 16])
def test_values_that_are_zero_or_constant(T):
    """Rows with scale 0 (all of one value) and rows of zeros, and keys to match."""
    c = Case([300], [T], T, 8, 2, 128, 64, seed=17)
    g = np.random.default_rng(18)
    L = 300 + T
    kv = g.standard_normal((2, L, 2, 128)).astype(np.float32)
    kv[1, :150] = 0.0
    kv[1, 150:200] = 2.5
    kv[0, 40:60] = 0.0
    kv[0, 250:] = -1.5
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[0]))
    c.K, c.V = [O.values(*O.quantise(kv[0]))], [O.values(*O.quantise(kv[1]))]
    c.check(c.run())
    kv[1] = 0.0
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[0]))
    assert (c.run() == 0).all()


@pytest.mark.parametrize("T", [1, 3, 16])
def test_rows_at_the_ends_of_the_range(T):
    """Keys and values of up to 3.3e38, whose |z| + 8 s passes the fp32 range, with
    queries that bring the scores back to ordinary size; then the smallest scales."""
    c = Case([300], [T], T, 10, 2, 128, 64, seed=19)
    g = np.random.default_rng(20)
    L = 300 + T
    kv = g.uniform(-1, 1, (2, L, 2, 128)).astype(np.float32)
    kv[1, 100:] += np.sign(kv[1, 100:, :, :1])   # rows with a centre of half the range
    kv[1] *= np.float32(0.5)
    for size in (3.3e38, 2.0 ** -96):
        x = kv * np.float32(size)
        c.cache.append(torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda(), to_dev_i32(c.slots[0]))
        c.K, c.V = [O.values(*O.quantise(x[0]))], [O.values(*O.quantise(x[1]))]
        q = np.float32(2.0 ** -100 if size > 1 else 2.0 ** 80)
        c.Q = torch.from_numpy(g.standard_normal((1, T, 10, 128)).astype(np.float32) * q).cuda().bfloat16()
        scale = float(np.float32(1 / size / q / 8))
        c.check(c.run(scale=scale, max_len=L), scale=scale)


@pytest.mark.parametrize("power", [-90, 101, 118])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_queries_at_the_ends_of_the_range(T, power):
    """Queries of 2^-90 and of 2^101 and 2^118 (products with the keys stay finite), the scale making up for it."""
    c = Case([260], [T], T, 10, 2, 128, 64, seed=21)
    f = float(2.0 ** power)
    c.Q = (c.Q.float() * f).bfloat16()
    scale = float(np.float32(128 ** -0.5 / f))
    c.check(c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("T,new", [(2, [0, 1, 2, 0]), (200, [0, 3, 200, 1])])
def test_rows_past_short_requests_where_most_of_the_gpu_is_idle(T, new):
    """A plan for long requests, a call with short ones: CTAs without work share in writing the zero rows."""
    c = Case([0, 5, 40, 130], new, T, 10, 2, 64, 16, seed=22)
    att = w12.KV4Attention(4, T, 10, 2, 64, 16, (len(c.table[0])) * 16)
    out = torch.full((4, T, 10, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = new_status()
    c.check(c.run(att=att, out=out, status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("T,d", [(1, 128), (17, 128), (17, 64)])
def test_rows_that_see_one_key_return_its_values(T, d):
    """The first token of an empty cache sees itself alone: every value of its key, those
    near 0 beside large ones among them, comes back to the roundings of that value."""
    c = Case([0] * 24, [T] * 24, T, 8, 2, d, 64, seed=23, std=3.0)
    out = c.run()
    c.check(out)
    out = out[:, 0].float().cpu().numpy().astype(np.float64).reshape(24, 2, 4, d)
    V = np.stack([v[0] for v in c.V])[:, :, None]
    assert (np.abs(out - V) <= np.abs(V) * (3 * U + 2.0 ** -12)).all()


@pytest.mark.parametrize("T,d", [(1, 128), (1, 64), (3, 128), (17, 128)])
@pytest.mark.parametrize("centre", [0.0, 1.0, 40.0])
def test_few_keys_of_large_spread(T, d, centre):
    """Two or three keys a request, scores far apart: outputs are small where the values of
    the key with the weight are, whatever the row's scale and centre."""
    c = Case([1, 2] * 40, [T] * 80, T, 8, 2, d, 16, seed=25)
    g = np.random.default_rng(26)
    for b in range(80):
        kv = (g.standard_normal((2, 1 + b % 2 + T, 2, d)) * 3).astype(np.float32)
        kv[1] += np.float32(centre * 3)
        c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[b]))
        c.K[b], c.V[b] = O.values(*O.quantise(kv[0])), O.values(*O.quantise(kv[1]))
    # Weights of less than 2^-14 round with 2^-25 of the largest: left out of the comparison
    # by scores that are no further apart than that.
    c.check(c.run(scale=0.01), scale=float(np.float32(0.01)))


def test_append_of_no_rows():
    c = Case([3], [1], 1, 2, 1, 64, 16, seed=24)
    before = c.cache.pool.clone()
    none = torch.from_numpy(np.zeros((0, 1, 64), dtype=np.float32)).cuda()
    for rows in (none, none.transpose(1, 2).contiguous().transpose(1, 2)):
        c.cache.append(rows, rows, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert torch.equal(c.cache.pool, before)


@pytest.mark.parametrize("T", [1, 16, 40])
def test_an_expired_wait_is_reported_and_the_next_call_is_right(T):
    """With a 1 us bound a wait may give up (W12_ERR_TIMEOUT); the call ends, and after
    the bound and the workspace are set back the next one matches the oracle."""
    c = Case([3000, 50], [T, T], T, 10, 2, 128, 64, seed=19)
    att = w12.KV4Attention(2, T, 10, 2, 128, 64, 3000 + T)
    torch.cuda.synchronize()
    w12.set_wait_limit_us(1)
    try:
        st = new_status()
        out = c.run(att=att, status=st)
        code = status_value(st)
    finally:
        w12.set_wait_limit_us(2000000)
    assert code in (0, 6)
    if code == 0:
        c.check(out)
    att.reset()
    st = new_status()
    c.check(c.run(att=att, status=st))
    assert status_value(st) == 0
