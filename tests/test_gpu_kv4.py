"""GPU rows of the paged 4-bit cache (append, read, commit) against the oracle.
Bytes are exact: every step of the quantiser is one IEEE fp32 operation."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")


def _cache(n_pages, Hkv, d, P, fill=0):
    c = w12.KV4Cache.create(n_pages, Hkv, d, P)
    c.pool.fill_(fill)
    return c


def _rows(n, Hkv, d, dtype, seed, wide=None, offset=0):
    """(K, V) views of a buffer whose rows are `wide` elements apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = Hkv * d
    wide = wide or 2 * width
    buf = (torch.randn((n, wide), generator=g, device="cuda") * 1.7 + 0.3).to(dtype)
    return (buf[:, offset:offset + width].unflatten(1, (Hkv, d)),
            buf[:, wide - width:].unflatten(1, (Hkv, d)))


def _check_append(n, Hkv, d, P, dtype, seed, slots, **kw):
    n_pages = max(slots) // P + 2
    c = _cache(n_pages, Hkv, d, P, fill=0xA5)
    K, V = _rows(n, Hkv, d, dtype, seed, **kw)
    before = c.pool.cpu().numpy()
    st = new_status()
    c.append(K, V, to_dev_i32(slots), status=st)
    assert status_value(st) == 0
    want = O.append(before, K.float().cpu().numpy(), V.float().cpu().numpy(), slots, d)
    assert (c.pool.cpu().numpy() == want).all()
    return c, slots


@pytest.mark.parametrize("n,Hkv,d,P", [(1, 1, 128, 16), (37, 3, 128, 64), (16, 8, 64, 32), (5, 2, 128, 128), (70, 1, 64, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_append_bytes(n, Hkv, d, P, dtype):
    g = np.random.default_rng(n)
    slots = g.permutation(n * 3)[:n].astype(int).tolist()
    slots[n // 2] = -1 if n > 1 else slots[0]
    c, slots = _check_append(n, Hkv, d, P, dtype, n + d, slots)
    K, V = c.read(to_dev_i32(slots))
    kr, vr = O.read(c.pool.cpu().numpy(), slots, d)
    for got, ref in ((K, kr), (V, vr)):
        # read rounds z + s (q - 8), one fp32 rounding, to bf16: the values of the oracle rounded the same way
        want = O._f32(O._bf16(ref.astype(np.float32)))
        assert (got.float().cpu().numpy() == want).all()


@pytest.mark.parametrize("dtype,wide,offset", [(torch.float32, 1000, 0), (torch.float32, 1001, 3), (torch.bfloat16, 777, 5),
                                               (torch.float16, 1024, 8), (torch.bfloat16, 1024, 1)])
def test_append_strided_and_unaligned_views(dtype, wide, offset):
    _check_append(9, 3, 128, 32, dtype, 5, list(range(20, 29)), wide=wide, offset=offset)


def test_append_reversed_and_broadcast_rows():
    """Negative strides cannot be had from torch; a broadcast row (stride 0) can."""
    c = _cache(2, 2, 64, 16)
    x = torch.randn((1, 2, 64), device="cuda").expand(4, 2, 64)
    c.append(x, x, to_dev_i32([0, 1, 2, 31]))
    K, V = c.read(to_dev_i32([0, 31]))
    assert (K[0] == K[1]).all() and (K == V).all() and (K != 0).any()


def test_append_special_rows():
    d, Hkv, P = 128, 1, 16
    x = np.zeros((7, 1, d), dtype=np.float32)
    x[1] = -2.25
    x[2, 0, 77] = np.inf
    x[3, 0, 3] = np.nan
    x[4, 0, ::2], x[4, 0, 1::2] = 3.3e38, -3.3e38
    x[5] = 1e-40
    x[6, 0, 0] = 1e-20
    c = _cache(1, Hkv, d, P)
    t = torch.from_numpy(x).cuda()
    c.append(t, t, to_dev_i32(range(7)))
    assert (c.pool.cpu().numpy() == O.append(np.zeros_like(c.pool.cpu().numpy()), x, x, range(7), d)).all()
    K, _ = c.read(to_dev_i32(range(7)))
    K = K.float().cpu().numpy()[:, 0]
    assert (K[0] == 0).all() and (K[1] == -2.25).all() and np.isnan(K[2:4]).all() and np.isfinite(K[4:]).all()


def test_slots_outside_the_pool_are_flagged_and_skipped():
    c = _cache(2, 1, 64, 16, fill=7)
    x = torch.randn((3, 1, 64), device="cuda")
    st = new_status()
    c.append(x, x, to_dev_i32([32, 5, -2]), status=st)
    assert status_value(st) == 1
    want = O.append(np.full((2, 1, 16 * 72), 7, dtype=np.uint8), x.cpu().numpy(), x.cpu().numpy(), [-1, 5, -1], 64)
    assert (c.pool.cpu().numpy() == want).all()
    st = new_status()
    K, V = c.read(to_dev_i32([1 << 30, 5, -1]), status=st)
    assert status_value(st) == 1 and (K[0] == 0).all() and (V[2] == 0).all() and (K[1] != 0).any()


def test_nothing_to_write_or_read():
    c = _cache(1, 2, 64, 16)
    x = torch.empty((0, 2, 64), device="cuda")
    c.append(x, x, torch.empty(0, dtype=torch.int32, device="cuda"))
    K, V = c.read(torch.empty(0, dtype=torch.int32, device="cuda"))
    assert K.shape == (0, 2, 64) and (c.pool == 0).all()


def test_a_pool_past_4_gigabytes():
    """Byte offsets pass 32 bits: rows of the first and last page."""
    d, Hkv, P = 128, 8, 128
    n_pages = (9 << 29) // (Hkv * P * (d + 8)) + 3      # 4.5 GiB and a little
    c = w12.KV4Cache(torch.empty((n_pages, Hkv, P * (d + 8)), dtype=torch.uint8, device="cuda"), P, d)
    K, V = _rows(4, Hkv, d, torch.bfloat16, 9)
    slots = [0, n_pages * P - 1, (n_pages - 1) * P, 5]
    c.append(K, V, to_dev_i32(slots))
    small = O.append(np.zeros((2, Hkv, P * (d + 8)), dtype=np.uint8), K.float().cpu().numpy(), V.float().cpu().numpy(),
                     [0, 2 * P - 1, P, 5], d)
    kr, vr = O.read(small, [0, 2 * P - 1, P, 5], d)
    Kg, Vg = c.read(to_dev_i32(slots))
    assert (Kg.float().cpu().numpy() == O._f32(O._bf16(kr.astype(np.float32)))).all()
    assert (Vg.float().cpu().numpy() == O._f32(O._bf16(vr.astype(np.float32)))).all()


@pytest.mark.parametrize("d,P,Hkv,layers", [(128, 16, 2, 1), (64, 32, 3, 3), (128, 64, 1, 70)])
def test_commit_matches_the_oracle(d, P, Hkv, layers):
    g = np.random.default_rng(d + P)
    B, T, max_pages = 4, 24, 6
    n_pages = B * max_pages
    table = g.permutation(n_pages).reshape(B, max_pages)
    prefix = np.array([0, P - 1, 2 * P + 3, 3 * P])
    path_len = np.array([1, 9, 4, 16])
    path = np.full((B, T), -1)
    for b in range(B):
        path[b, :path_len[b]] = np.sort(g.permutation(T)[:path_len[b]])
    path[2, :4] = [0, 1, 2, 3]                          # a block's prefix: nothing moves
    pools = [g.integers(0, 256, (n_pages, Hkv, P * (d + 8))).astype(np.uint8) for _ in range(min(layers, 3))]
    caches = [w12.KV4Cache(torch.from_numpy(pools[i % len(pools)]).cuda(), P, d) for i in range(layers)]
    st = new_status()
    new = w12.kv4_commit(caches, to_dev_i32(table), to_dev_i32(prefix), to_dev_i32(path), to_dev_i32(path_len), status=st)
    assert status_value(st) == 0
    assert new.cpu().tolist() == (prefix + path_len).tolist()
    for i in (0, layers // 2, layers - 1):
        want = O.commit(pools[i % len(pools)], table, prefix, path, path_len, d)
        assert (caches[i].pool.cpu().numpy() == want).all()


@pytest.mark.parametrize("path,n,prefix,table", [([1, 0], 2, 0, [0, 1]), ([0, 0], 2, 0, [0, 1]), ([0, 1], 0, 0, [0, 1]), ([0, 1], 3, 0, [0, 1]),
                                                 ([0, 40], 2, 0, [0, 1]), ([0, 17], 2, 0, [0, -1]), ([0, 17], 2, 0, [0, 9]), ([0, 1], 2, -1, [0, 1])])
def test_commit_leaves_a_request_with_a_bad_path(path, n, prefix, table):
    g = np.random.default_rng(1)
    pool = g.integers(0, 256, (2, 1, 16 * 72)).astype(np.uint8)
    c = w12.KV4Cache(torch.from_numpy(pool).cuda(), 16, 64)
    st = new_status()
    new = w12.kv4_commit([c], to_dev_i32([table]), to_dev_i32([prefix]), to_dev_i32([path]), to_dev_i32([n]), status=st)
    assert status_value(st) == 4 and new.item() == prefix
    assert (c.pool.cpu().numpy() == pool).all()


def test_binding_refusals():
    c = _cache(2, 2, 64, 16)
    x = torch.zeros((3, 2, 64), device="cuda")
    s = to_dev_i32([0, 1, 2])
    with pytest.raises(TypeError):
        c.append(x.double(), x.double(), s)
    with pytest.raises(TypeError):
        c.append(x, x.half(), s)
    with pytest.raises(ValueError):
        c.append(x[:, :1], x[:, :1], s)
    with pytest.raises(ValueError):
        c.append(x, x, s[:2])
    with pytest.raises(ValueError):
        c.append(x.transpose(1, 2).contiguous().transpose(1, 2), x, s)
    with pytest.raises(ValueError):
        c.append(x.cpu(), x, s)
    with pytest.raises(ValueError):
        c.read(s.long())
    with pytest.raises(ValueError):
        w12.KV4Cache(torch.zeros((2, 2, 16 * 72), dtype=torch.uint8, device="cuda"), 16, 128)
    one = to_dev_i32([0])
    with pytest.raises(ValueError):
        w12.kv4_commit([c], to_dev_i32([[0, 1]]), one, to_dev_i32([[0, 1]]), to_dev_i32([1]), new_len=one)
    with pytest.raises(w12.W12Error) as e:
        w12.kv4_commit([c, _cache(2, 2, 128, 16)], to_dev_i32([[0, 1]]), one, to_dev_i32([[0, 1]]), to_dev_i32([1]))
    assert e.value.code == 2
