"""How near attention over the paged 4-bit cache comes to its definition, on both sides
of the rule between its two kernels (up to 16 rows a kv head, and more).

The bounds count the roundings that include/w12.h promises (fp16 operands, half a
step: 2^-11 relative) and one bf16 rounding of the output (2^-8), nothing looser:

  keys      2^-11 |K| a value, or 2^-16 of 8/7 of its row's largest where that is more
            (8/7: |z| + 8 s over the largest |z + s (q - 8)|). A row's scores move by at
            most D = scale max_j sum_c |q_c| (2^-11 |K_jc| + 2^-16 8/7 max |K_j|), its
            weights by a factor within e^(2 D)
  weights   2^-11 relative, or 2^-30 of the row's largest weight times value row
  values    2^-11 |V|, or 2^-16 of 8/7 of the value row's largest
  fp32 sums and exponentials of scores below 2^8: 2^-14
  output    2^-8 of itself

Over a whole output these are independent. bf16's rounding of values of spread mantissas
is 1.5e-3 to 1.7e-3 of the norm, each fp16 rounding at most 2^-11 / sqrt(3) = 2.8e-4, so
their root sum of squares is below 1.8e-3; the limit is 2^-9 = 1.95e-3. One operand in
bf16 would make it 2.3e-3.
"""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as O
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")

H = 2.0 ** -11       # a rounding to fp16
ROW = 2.0 ** -16 * 8 / 7
NORM = 2.0 ** -9


def fill(c, b, kv):
    """Request b's rows [2, L, Hkv, d] in place of the ones it has."""
    kv = np.ascontiguousarray(kv, dtype=np.float32)
    c.cache.append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(), to_dev_i32(c.slots[b]))
    c.K[b], c.V[b] = O.values(*O.quantise(kv[0])), O.values(*O.quantise(kv[1]))


def check(c, out, scale=None, rows=None):
    """out against float64 for the (request, token) pairs in rows (default: all)."""
    scale = float(np.float32(c.d ** -0.5 if scale is None else scale))
    out = out.float().cpu().numpy().astype(np.float64)
    Q = c.Q.float().cpu().numpy().astype(np.float64)
    G = c.Hq // c.Hkv
    err2 = ref2 = 0.0
    for b in range(c.B):
        n = c.new[b]
        see = O.visible(c.prefix[b], n, None if c.parents is None else c.parents[b])
        for t in range(n):
            if rows is not None and (b, t) not in rows:
                continue
            at = np.nonzero(see[t])[0]
            for h in range(c.Hkv):
                q, K, V = Q[b, t, h * G:(h + 1) * G], c.K[b][at, h], c.V[b][at, h]
                s = scale * (q @ K.T)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                ref, A = p @ V, p @ np.abs(V)
                Kmax, Vmax = np.abs(K).max(1), np.abs(V).max(1)
                D = scale * (H * (np.abs(q) @ np.abs(K).T) + ROW * np.abs(q).sum(1)[:, None] * Kmax).max(1, keepdims=True)
                bound = A * (np.expm1(2 * D) + 2 * H + 2.0 ** -14) + ROW * (p @ Vmax)[:, None] \
                    + 2.0 ** -30 * len(at) * (p * Vmax).max(1)[:, None] + 2.0 ** -8 * np.abs(ref) + 1e-36
                err = out[b, t, h * G:(h + 1) * G] - ref
                assert np.isfinite(err).all(), (b, t, h)
                worst = np.unravel_index(np.argmax(np.abs(err) - bound), err.shape)
                assert (np.abs(err) <= bound).all(), f"b={b} t={t} h={h} {worst}: {err[worst]} above {bound[worst]}"
                err2 += (err ** 2).sum()
                ref2 += (ref ** 2).sum()
    rel = (err2 / ref2) ** 0.5
    assert rel <= NORM, f"relative error {rel}"
    return rel


# (T, Hq, Hkv): 1, 5, 8, 12, 16 rows a kv head; then 17, 20, 80 and two tiles.
SHAPES = [(1, 2, 2), (1, 10, 2), (2, 8, 2), (3, 8, 2), (4, 8, 2), (17, 2, 2), (5, 8, 2), (16, 10, 2), (40, 8, 2)]


@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_ordinary_rows(T, Hq, Hkv, d, tree):
    c = Case([900, 77], [T, T], T, Hq, Hkv, d, 32, seed=T + d)
    if tree and T > 1:
        c.trees(T)
    st = new_status()
    check(c, c.run(status=st))
    assert status_value(st) == 0


@pytest.mark.parametrize("T,Hq,Hkv", [(4, 8, 2), (5, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("power", [8, 18, 22, 26, 60])
@pytest.mark.parametrize("which", ["key", "value", "both"])
@pytest.mark.parametrize("tree", [False, True])
def test_a_large_row_in_a_masked_place(T, Hq, Hkv, power, which, tree):
    """The last new token's key or value row is 2^power times the others'. The tokens that
    do not see it answer as if it were not there."""
    c = Case([150], [T], T, Hq, Hkv, 128, 64, seed=31)
    if tree:
        c.trees(4)
    g = np.random.default_rng(32)
    kv = g.standard_normal((2, 150 + T, Hkv, 128)).astype(np.float32)
    for i, name in enumerate(("key", "value")):
        if which in (name, "both"):
            kv[i, -1] *= np.float32(2.0 ** power)
    fill(c, 0, kv)
    check(c, c.run(), rows={(0, t) for t in range(T - 1)})


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (5, 8, 2)])
@pytest.mark.parametrize("power", [7, 20, 30])
def test_large_values_without_weight(T, Hq, Hkv, power):
    """Every seventh key has a value row 2^power times the others' and next to no weight."""
    d = 128
    c = Case([700], [T], T, Hq, Hkv, d, 64, seed=33)
    g = np.random.default_rng(34)
    c.Q = torch.from_numpy((1 + 0.1 * g.standard_normal((1, T, Hq, d))).astype(np.float32)).cuda().bfloat16()
    kv = g.standard_normal((2, 700 + T, Hkv, d)).astype(np.float32)
    kv[0] *= 0.1
    kv[0, :700:7] -= np.float32(60 / d ** 0.5)        # scores of about -60
    kv[1, :700:7] *= np.float32(2.0 ** power)
    fill(c, 0, kv)
    check(c, c.run())


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (5, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("gap", [14, 16])
@pytest.mark.parametrize("value", [0.0, 1e-6])
@pytest.mark.parametrize("apart", [False, True])
def test_a_dominant_key_with_a_small_value_row(T, Hq, Hkv, gap, value, apart):
    """One key (the first, or one among the others) scores `gap` nats above all others
    and adds nothing to the output, which is then the others' alone."""
    d, L = 128, 3000
    c = Case([L], [T], T, Hq, Hkv, d, 64, seed=35)
    g = np.random.default_rng(36)
    c.Q = torch.from_numpy((1 + 0.02 * g.standard_normal((1, T, Hq, d))).astype(np.float32)).cuda().bfloat16()
    kv = g.standard_normal((2, L + T, Hkv, d)).astype(np.float32)
    kv[0] *= 0.05
    at = 1717 if apart else 0
    kv[0, at] = np.float32(gap / d ** 0.5)
    kv[1, at] *= np.float32(value)
    fill(c, 0, kv)
    check(c, c.run())


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (5, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("gap", [12, 16])
def test_a_dominant_key_whose_values_are_zero_in_some_dims(T, Hq, Hkv, gap):
    """Where the value row of a key `gap` nats above the others is zero, the output is the
    others' alone; elsewhere it is that key's."""
    d, L = 128, 3000
    c = Case([L], [T], T, Hq, Hkv, d, 64, seed=37)
    g = np.random.default_rng(38)
    c.Q = torch.from_numpy((1 + 0.02 * g.standard_normal((1, T, Hq, d))).astype(np.float32)).cuda().bfloat16()
    kv = g.standard_normal((2, L + T, Hkv, d)).astype(np.float32)
    kv[0] *= 0.05
    kv[0, 5] = np.float32(gap / d ** 0.5)
    kv[1, 5] = np.float32(15 / 64) * (np.arange(d) % 2)
    fill(c, 0, kv)
    assert (c.V[0][5, :, ::2] == 0).all() and (c.V[0][5, :, 1::2] == 15 / 64).all()
    check(c, c.run())
    if T * Hq // Hkv <= 16:
        return  # there p s (q - 8) and p z are summed apart in fp32: 2^-24 of the key's 8 s is 1e-3 of these
    # The dims of the others alone, over all rows together.
    K, V, q = c.K[0][:, 0], c.V[0][:, 0, ::2], c.Q[0, :, 0].float().cpu().numpy().astype(np.float64)
    out = c.run()[0, :, 0, ::2].float().cpu().numpy().astype(np.float64)
    err2 = ref2 = 0.0
    for t in range(T):
        s = d ** -0.5 * (K[:L + t + 1] @ q[t])
        p = np.exp(s - s.max())
        ref = p @ V[:L + t + 1] / p.sum()
        err2 += ((out[t] - ref) ** 2).sum()
        ref2 += (ref ** 2).sum()
    assert (err2 / ref2) ** 0.5 <= NORM


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (5, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("power", [40, 60, 80])
def test_blocks_of_zero_values_beside_very_large_ones(T, Hq, Hkv, power):
    """Runs of keys with most of the weight and value rows of zeros, beside value rows of
    2^power: their weight stays in the denominator."""
    d, L = 128, 500
    c = Case([L], [T], T, Hq, Hkv, d, 64, seed=39)
    g = np.random.default_rng(40)
    c.Q = torch.from_numpy((1 + 0.1 * g.standard_normal((1, T, Hq, d))).astype(np.float32)).cuda().bfloat16()
    kv = g.standard_normal((2, L + T, Hkv, d)).astype(np.float32)
    kv[0] *= 0.1
    kv[0, 128:256] += np.float32(6 / d ** 0.5)
    kv[1] *= np.float32(2.0 ** power)
    kv[1, 128:256] = 0.0
    fill(c, 0, kv)
    check(c, c.run())


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (5, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("power", [-60, -50, -44, -40])
def test_small_values_of_varied_size(T, Hq, Hkv, power):
    """Value rows of 2^power to 2^(power + 6), all of them small."""
    c = Case([300], [T], T, Hq, Hkv, 128, 64, seed=41)
    g = np.random.default_rng(42)
    kv = g.standard_normal((2, 300 + T, Hkv, 128)).astype(np.float32)
    kv[1] *= np.float32(2.0 ** power) * (np.float32(2.0) ** g.integers(0, 7, (300 + T, 1, 1))).astype(np.float32)
    fill(c, 0, kv)
    check(c, c.run())
