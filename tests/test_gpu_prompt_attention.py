"""Causal attention over packed prompts on the GPU against the float64 oracle.

An output is off by its own rounding (u = 2^-8 of it in bf16, 2^-11 in fp16), by the weights'
roundings (u of sum p |V|; in fp16 also 2^-25 of the largest weight for each key: 2^-25 sum |V|, the
largest weight being 1 or more and so the denominator), and by the scores' (fp32 sums of d
products, at most d 2^-24 of scale |q|.|K|, in the weight and in the denominator) and the
exponential's (2^-22, twice), both relative to sum p |V|. Sums over the keys in fp32 add
2^-20 of it (128 keys a matrix product's accumulation, joined block by block)."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import layer_oracle as O
from speculative_decoding_verification_w12_gb300 import w12

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _offsets(lens, first=0):
    return (first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int64)


def _rows(total, Hq, Hkv, d, dtype, seed, strided=False, extra=8, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = (torch.randn((total, (Hq + 2 * Hkv) * d + extra), generator=g, device="cuda") * scale).to(dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in wide[:, :(Hq + 2 * Hkv) * d].split([Hq * d, Hkv * d, Hkv * d], 1))
    return (q, k, v) if strided else tuple(x.contiguous() for x in (q, k, v))


def _close(got, q, k, v, cu, scale):
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    o, a, e, s = O.prompt_attention(f(q), f(k), f(v), cu, scale)
    rows = np.concatenate([np.arange(x, y) for x, y in zip(cu[:-1], cu[1:])]) if len(cu) > 1 else np.arange(0)
    rows = rows.astype(int)
    u = 2.0 ** -8 if got.dtype is BF16 else 2.0 ** -11
    tol = u * np.abs(o) + (u + 2 * q.shape[2] * 2.0 ** -24 * e[..., None] + 2.0 ** -19) * (1 + u) * a
    if got.dtype is F16:
        tol = tol + 2.0 ** -25 * s + 2.0 ** -25
    err = np.abs(f(got)[rows].astype(np.float64) - o[rows])
    assert np.isfinite(f(got)[rows]).all()
    assert (err <= tol[rows]).all(), (err / tol[rows]).max()


LENS = [[1], [2], [25], [127], [128], [129], [777], [0, 1, 0, 3], [50, 51, 25, 26, 1], [300, 0, 1, 257, 40]]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, d, dtype):
    cu = _offsets(lens)
    q, k, v = _rows(cu[-1], 10, 2, d, dtype, len(lens))
    st = new_status()
    o = w12.prompt_attention(q, k, v, to_dev_i32(cu), status=st)
    assert status_value(st) == 0 and o.dtype is dtype and o.shape == q.shape
    _close(o, q, k, v, cu, d ** -0.5)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (2, 1), (12, 4), (8, 2), (40, 8), (14, 2), (16, 1), (33, 1), (128, 1)])
def test_groups_of_heads(Hq, Hkv):
    cu = _offsets([70, 1, 200, 33])
    q, k, v = _rows(cu[-1], Hq, Hkv, 64, BF16, Hq, strided=True)
    _close(w12.prompt_attention(q, k, v, to_dev_i32(cu)), q, k, v, cu, 0.125)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [([2100], 5, 1, 128), ([1500, 900], 4, 2, 64), ([1300, 5, 0, 640], 3, 3, 128)])
def test_longer_prompts_as_views(lens, Hq, Hkv, d, dtype):
    cu = _offsets(lens)
    q, k, v = _rows(cu[-1], Hq, Hkv, d, dtype, 9, strided=True)
    _close(w12.prompt_attention(q, k, v, to_dev_i32(cu)), q, k, v, cu, d ** -0.5)


def test_many_sequences():
    """More sequences than a warp has lanes, of lengths on both sides of a tile's."""
    g = np.random.default_rng(0)
    cu = _offsets(g.choice([0, 1, 2, 30, 63, 64, 65, 127, 128, 130, 200], 150))
    q, k, v = _rows(cu[-1], 4, 2, 64, BF16, 3)
    st = new_status()
    o = w12.prompt_attention(q, k, v, to_dev_i32(cu), status=st)
    assert status_value(st) == 0
    _close(o, q, k, v, cu, 0.125)


def test_rows_outside_the_sequences_are_left_as_they_are():
    cu = _offsets([40, 0, 90], first=7)
    q, k, v = _rows(200, 4, 2, 128, BF16, 3)
    out = torch.full_like(q, 5.0)
    o = w12.prompt_attention(q, k, v, to_dev_i32(cu), out=out)
    assert o is out and (out[:7] == 5).all() and (out[cu[-1]:] == 5).all()
    _close(out, q, k, v, cu, 128 ** -0.5)


def test_no_tokens_and_no_sequences():
    q, k, v = _rows(8, 4, 2, 64, BF16, 3)
    out = torch.full_like(q, 5.0)
    for cu in ([0], [0, 0], [8, 8, 8]):
        st = new_status()
        w12.prompt_attention(q, k, v, to_dev_i32(cu), out=out, status=st)
        assert status_value(st) == 0 and (out == 5).all()
    assert w12.prompt_attention(q[:0], k[:0], v[:0], to_dev_i32([0, 0])).shape == (0, 4, 64)


@pytest.mark.parametrize("cu", [[0, 20, 10, 30], [0, -3, 10, 30], [-5, 4, 10, 30], [0, 10, 31, 31]])
def test_offsets_out_of_range(cu):
    q, k, v = _rows(30, 4, 2, 64, BF16, 3)
    out = torch.full_like(q, 5.0)
    st = new_status()
    w12.prompt_attention(q, k, v, to_dev_i32(cu), out=out, status=st)
    assert status_value(st) == 1
    good = [(a, e) for a, e in zip(cu, cu[1:]) if 0 <= a <= e <= 30]
    times = np.zeros(30, dtype=int)                      # (rows of two sequences get either's result)
    for a, e in good:
        times[a:e] += 1
    for a, e in good:
        part = w12.prompt_attention(q[a:e], k[a:e], v[a:e], to_dev_i32([0, e - a]))
        once = torch.from_numpy(times[a:e] == 1).cuda()
        assert torch.equal(out[a:e][once], part[once])
    assert (out[torch.from_numpy(times == 0).cuda()] == 5).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,d", [(5, 1, 128), (4, 2, 64), (1, 1, 128)])
def test_masked_places_may_hold_anything(Hq, Hkv, d, dtype):
    """Keys and values that are not finite reach the rows that see them and no other."""
    lens = [300, 40, 130]
    cu = _offsets(lens)
    q, k, v = _rows(cu[-1] + 30, Hq, Hkv, d, dtype, 4)
    clean = w12.prompt_attention(q, k, v, to_dev_i32(cu))
    nan, inf = float("nan"), float("inf")
    for values, keys in ((True, False), (False, True), (True, True)):
        qq, kk, vv = q.clone(), k.clone(), v.clone()
        bad = {0: [270, 299], 1: [39], 2: [0, 129]}      # places in the sequences
        kk[cu[-1]:], vv[cu[-1]:], qq[cu[-1]:] = nan, inf, nan  # rows behind the last sequence
        hit = torch.zeros(len(q), dtype=torch.bool, device="cuda")
        for b, places in bad.items():
            for n, p in enumerate(places):
                if values:
                    vv[cu[b] + p, 0, n::3] = (inf, nan, -inf)[(n + b) % 3]
                if keys:
                    kk[cu[b] + p, 0, 5] = (nan, inf)[n % 2]
                hit[cu[b] + p:cu[b + 1]] = True
        out = torch.full_like(qq, 5.0)
        st = new_status()
        w12.prompt_attention(qq, kk, vv, to_dev_i32(cu), out=out, status=st)
        assert status_value(st) == 0
        whole = torch.arange(len(q), device="cuda") < int(cu[-1])
        assert torch.equal(out[whole & ~hit], clean[whole & ~hit])
        assert (out[~whole] == 5).all()
        if values:                                        # every row that sees one has it
            last = hit & whole
            assert not torch.isfinite(out[last][:, 0]).all(-1).any()
        if values and not keys:                           # in its columns alone, and with its sign
            for b, places in bad.items():
                n, p = 0, places[0]
                col = vv[cu[b] + p, 0, 0].item()
                got = out[cu[b] + p, 0]
                assert (torch.isnan(got[0::3]) if col != col else got[0::3] == col).all()
                assert torch.equal(got[1::3], clean[cu[b] + p, 0][1::3]) and torch.equal(got[2::3], clean[cu[b] + p, 0][2::3])


def test_a_query_that_is_not_finite_and_keys_of_minus_infinity():
    cu = _offsets([200])
    q, k, v = _rows(200, 2, 1, 64, BF16, 4)
    clean = w12.prompt_attention(q, k, v, to_dev_i32(cu))
    q[60, 1, 3] = float("nan")
    o = w12.prompt_attention(q, k, v, to_dev_i32(cu))
    assert torch.isnan(o[60, 1]).all()
    o[60, 1] = clean[60, 1]
    assert torch.equal(o, clean)
    q[:] = 1.0
    k[0] = float("-inf")                                  # every row sees it: weighs nothing; row 0 sees no other
    o = w12.prompt_attention(q, k, v, to_dev_i32(cu))
    assert (o[0] == 0).all() and torch.isfinite(o).all()
    rest = w12.prompt_attention(q[1:].contiguous(), k[1:].contiguous(), v[1:].contiguous(), to_dev_i32([0, 199]))
    assert (o[1:].float() - rest.float()).abs().max() <= 2.0 ** -6 * v.float().abs().max()


@pytest.mark.parametrize("scale_of", [1e-4, 6.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_flat_and_peaked_weights(scale_of, dtype):
    cu = _offsets([513])
    q, k, v = _rows(513, 4, 2, 64, dtype, 6, scale=scale_of ** 0.5)
    _close(w12.prompt_attention(q, k, v, to_dev_i32(cu), scale=0.5), q, k, v, cu, 0.5)


def test_maxima_that_climb_block_by_block():
    """Later keys outweigh all before them by more than any weight's range: sums and outputs are rescaled."""
    cu = _offsets([700])
    q, k, v = _rows(700, 2, 1, 128, BF16, 6)
    q[:] = 1.0
    k[:] = (torch.arange(700, device="cuda") // 100 * 4.0)[:, None, None].to(BF16)
    _close(w12.prompt_attention(q, k, v, to_dev_i32(cu)), q, k, v, cu, 128 ** -0.5)
    k[:] = -k
    _close(w12.prompt_attention(q, k, v, to_dev_i32(cu)), q, k, v, cu, 128 ** -0.5)


def test_graph_side_stream_and_the_same_bits():
    cu = _offsets([150, 60, 3])
    q, k, v = _rows(230, 10, 2, 128, BF16, 6)
    dev = to_dev_i32(cu)
    first = w12.prompt_attention(q, k, v, dev, out=torch.zeros_like(q))
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w12.prompt_attention(q, k, v, dev, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    cu = _offsets([10, 200, 20])
    dev.copy_(to_dev_i32(cu))
    g.replay()
    torch.cuda.synchronize()
    _close(out, q, k, v, cu, 128 ** -0.5)
    side = torch.cuda.Stream()
    again = w12.prompt_attention(q, k, v, dev, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


def test_an_expired_wait_is_reported_and_the_next_call_is_whole():
    cu = _offsets([1900, 2000])
    q, k, v = _rows(3900, 40, 8, 128, BF16, 6)
    want = w12.prompt_attention(q, k, v, to_dev_i32(cu))
    st = new_status()
    w12.set_wait_limit_us(1)
    try:
        w12.prompt_attention(q, k, v, to_dev_i32(cu), status=st)
        torch.cuda.synchronize()
    finally:
        w12.set_wait_limit_us(2000000)
    assert status_value(st) in (0, 6)
    assert torch.equal(w12.prompt_attention(q, k, v, to_dev_i32(cu)), want)


def test_rows_past_32_bits():
    """Rows 2^23 values apart, 600 of them (an infinity among the values); more than 2^31 outputs."""
    n, apart = 600, 2 ** 23
    base = torch.empty(n * apart, dtype=BF16, device="cuda")
    q, k, v = (base.as_strided((n, h, 128), (apart, 128, 1), at) for h, at in ((4, 0), (2, 512), (2, 768)))
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    v[599, 1, 7] = float("inf")
    cu, st = to_dev_i32([0, 90, n]), new_status()
    got = w12.prompt_attention(q, k, v, cu, status=st)
    want = w12.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(got, want) and torch.isinf(got[599, 2:, 7]).all() and torch.isfinite(got[:599]).all()
    del base, q, k, v
    L, B, H = 300, 900, 64
    q, k, v = (torch.randn((L * B, h, 128), generator=g, device="cuda", dtype=BF16) for h in (H, 8, 8))
    assert q.numel() > 2 ** 31
    out = w12.prompt_attention(q, k, v, to_dev_i32(np.arange(B + 1) * L), status=st)
    for b in (0, B // 2, B - 1):
        one = slice(b * L, b * L + L)
        assert torch.equal(out[one], w12.prompt_attention(q[one], k[one], v[one], to_dev_i32([0, L])))
    assert status_value(st) == 0


def test_calls_at_the_same_time():
    """Two streams at once, each with calls of its own sizes: what each gives alone."""
    cases = []
    for lens, Hq, Hkv, d, dtype in (([700, 33], 8, 2, 128, BF16), ([130, 1, 500], 4, 4, 64, F16)):
        q, k, v = _rows(sum(lens), Hq, Hkv, d, dtype, len(lens))
        cases.append((q, k, v, to_dev_i32(_offsets(lens))))
    alone = [w12.prompt_attention(*c) for c in cases]
    streams, got, st = [torch.cuda.Stream() for _ in cases], [[] for _ in cases], new_status()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, g in zip(cases, streams, got):
            g.append(w12.prompt_attention(*c, status=st, stream=s))
    torch.cuda.synchronize()
    assert status_value(st) == 0
    assert all(torch.equal(x, want) for g, want in zip(got, alone) for x in g)


@pytest.mark.parametrize("lens", ["ragged", "long and short"])
def test_groups_of_sequences(lens):
    """More keys and values than one group of sequences has, over several of the walk's chunks: each
    sequence bitwise as it comes by itself."""
    rng = np.random.default_rng(5)
    lens = [int(v) for v in (rng.integers(0, 500, 70) if lens == "ragged" else rng.permutation([2200, 1900, 1500] + [3] * 60 + [0] * 5))]
    H, d = 64, 128
    cu, total = _offsets(lens), sum(lens)
    assert 4 * total * H * d > 4 * 43 * 2 ** 20
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((total, H, d), generator=g, device="cuda", dtype=BF16) for _ in range(3))
    st = new_status()
    out = w12.prompt_attention(q, k, v, to_dev_i32(cu), out=torch.full_like(q, float("nan")), status=st)
    assert status_value(st) == 0
    for a, e in zip(cu[:-1], cu[1:]):
        if e > a:
            assert torch.equal(out[a:e], w12.prompt_attention(q[a:e], k[a:e], v[a:e], to_dev_i32([0, e - a]))), (a, e)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 5, 16])
def test_two_tiles_an_item_give_what_one_gives(G, d, dtype):
    """Sixteen kv heads fill the GPU with items of two tiles; each by itself leaves it to single ones. With
    values and keys that are not finite here and there."""
    lens = [300, 0, 1, 257, 40, 513, 79, 80, 81, 128, 16]
    cu, Hkv = _offsets(lens), 16
    q, k, v = _rows(sum(lens), Hkv * G, Hkv, d, dtype, G + d)
    for i, bad in enumerate((float("inf"), float("nan"), float("-inf"))):
        v[37 + 211 * i, i, 5] = bad
        v[301 + 17 * i, 4 + i, d - 1] = bad
        k[640 + 30 * i, 8 + i, 3] = bad
    dev, st = to_dev_i32(cu), new_status()
    out = w12.prompt_attention(q, k, v, dev, status=st)
    assert status_value(st) == 0
    for h in range(Hkv):
        heads = slice(h * G, h * G + G)
        one = w12.prompt_attention(q[:, heads], k[:, h:h + 1], v[:, h:h + 1], dev)
        assert torch.equal(torch.nan_to_num(out[:, heads], 77.0), torch.nan_to_num(one, 77.0)), h
        assert torch.equal(torch.isnan(out[:, heads]), torch.isnan(one)), h
    clean = slice(11 * G, 16 * G)                          # heads without such values
    _close(out[:, clean], q[:, clean], k[:, 11:], v[:, 11:], cu, d ** -0.5)
