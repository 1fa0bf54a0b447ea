"""Low-rank adapters beside a projection on the GPU against the float64 oracle.

Products of bf16 numbers are exact; a matrix instruction adds 16 of them and the sum so far with
an error of at most 2^-20 of their sizes (16 additions of 2^-24). A row's sum passes through
2 ceil(K / 2048) of them and twelve fp32 additions, the second product through 3 ceil(r / 16) (its T is
whole to 2^-24), and Y's addition rounds once: in all (2 ceil(K/2048) + 3 ceil(r/16) + 2) 2^-20 of
scale |B| |A| |x|, and 2^-24 of the result."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import layer_oracle as O
from speculative_decoding_verification_w12_gb300 import w12

pytestmark = pytest.mark.gpu


def _make(n, N, K, r, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = (torch.randn((n, r, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    B = torch.randn((n, N, r), generator=g, device="cuda").bfloat16()
    return A, B, torch.rand(n, generator=g, device="cuda") + 0.5, g


def _check(X, Y0, Y, A, B, scale, ids):
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    want, most = O.lora(f(X), f(Y0), f(A), f(B), f(scale), ids)
    K, r = A.shape[2], A.shape[1]
    tol = (2 * -(-K // 2048) + 3 * -(-r // 16) + 2) * 2.0 ** -20 * most + 2.0 ** -24 * np.abs(want)
    err = np.abs(f(Y).astype(np.float64) - want)
    assert (err <= tol).all(), (err - tol).max()
    idle = [m for m, a in enumerate(ids) if a < 0]
    assert torch.equal(Y[idle], Y0[idle])


@pytest.mark.parametrize("M,N,K,r,n,ids", [
    (1, 16, 8, 8, 1, "same"), (16, 512, 512, 16, 3, "same"), (17, 528, 520, 16, 3, "same"), (64, 128, 1024, 24, 5, "mixed"),
    (64, 640, 264, 32, 128, "each"), (256, 256, 2056, 64, 7, "mixed"), (256, 1040, 512, 128, 256, "each"), (33, 5120, 5120, 16, 2, "idle"),
    (200, 48, 4096, 48, 16, "blocks"), (256, 128, 136, 8, 1, "same"), (5, 2064, 17408, 128, 4, "mixed"), (40, 64, 64, 104, 3, "none")])
def test_against_the_oracle(M, N, K, r, n, ids):
    A, B, scale, g = _make(n, N, K, r)
    rng = np.random.default_rng(M)
    which = {"same": [n - 1] * M, "mixed": rng.integers(0, n, M), "each": rng.permutation(n)[:M], "idle": rng.integers(-1, n, M),
             "blocks": np.repeat(rng.integers(-1, n, -(-M // 16)), 16)[:M], "none": [-1] * M}[ids]
    which = [int(a) for a in which]
    X, Y0 = torch.randn((M, K), generator=g, device="cuda").bfloat16(), torch.randn((M, N), generator=g, device="cuda")
    Y = Y0.clone()
    st = new_status()
    lora = w12.LoRA(A, B, scale, max_rows=M)
    assert lora.run(X, Y, to_dev_i32(which), status=st) is Y
    assert status_value(st) == 0
    _check(X, Y0, Y, A, B, scale, which)
    # The same inputs give the same bits.
    again = Y0.clone()
    lora.run(X, again, to_dev_i32(which))
    assert torch.equal(again, Y)


def test_padded_rows_and_what_lies_between_them():
    A, B, scale, g = _make(3, 64, 72, 16)
    wide_x, wide_y = torch.randn((20, 88), generator=g, device="cuda").bfloat16(), torch.randn((20, 100), generator=g, device="cuda")
    before = wide_y.clone()
    X, Y = wide_x[:, 8:80], wide_y[:, 4:68]
    ids = [m % 4 - 1 for m in range(20)]
    w12.LoRA(A, B, scale).run(X, Y, to_dev_i32(ids))
    _check(X, before[:, 4:68], Y, A, B, scale, ids)
    assert torch.equal(wide_y[:, :4], before[:, :4]) and torch.equal(wide_y[:, 68:], before[:, 68:])


def test_ids_out_of_range_are_taken_for_none():
    A, B, scale, g = _make(3, 64, 64, 16)
    X, Y0 = torch.randn((4, 64), generator=g, device="cuda").bfloat16(), torch.randn((4, 64), generator=g, device="cuda")
    for bad in (3, -2, 2 ** 31 - 1, -2 ** 31):
        Y, st = Y0.clone(), new_status()
        w12.LoRA(A, B, scale).run(X, Y, to_dev_i32([0, bad, 2, -1]), status=st)
        assert status_value(st) == 1
        _check(X, Y0, Y, A, B, scale, [0, -1, 2, -1])


def test_one_workspace_for_batches_of_any_size_and_a_graph():
    A, B, scale, g = _make(40, 96, 256, 32)
    lora = w12.LoRA(A, B, scale)
    rng = np.random.default_rng(1)
    for M in (256, 1, 77, 16, 256):
        ids = rng.integers(-1, 40, M).tolist()
        X, Y0 = torch.randn((M, 256), generator=g, device="cuda").bfloat16(), torch.randn((M, 96), generator=g, device="cuda")
        Y = Y0.clone()
        lora.run(X, Y, to_dev_i32(ids))
        _check(X, Y0, Y, A, B, scale, ids)
    dev_ids = to_dev_i32([0] * 16)
    X, Y = torch.randn((16, 256), generator=g, device="cuda").bfloat16(), torch.zeros((16, 96), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lora.run(X, Y, dev_ids)
    ids = [3, 3, -1, 7] * 4
    dev_ids.copy_(to_dev_i32(ids))
    Y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    _check(X, torch.zeros_like(Y), Y, A, B, scale, ids)
    side = torch.cuda.Stream()
    Z = torch.zeros_like(Y)
    torch.cuda.synchronize()
    lora.run(X, Z, dev_ids, stream=side)
    side.synchronize()
    assert torch.equal(Z, Y)


def test_sizes_and_values_at_the_ends():
    """Large and tiny adapters, and rows that are not finite: those rows alone are so after."""
    A, B, scale, g = _make(2, 32, 64, 8)
    scale.fill_(1.0)
    X = torch.randn((6, 64), generator=g, device="cuda").bfloat16()
    X[0] *= 1e30
    X[1] *= 1e-30
    Y0 = torch.zeros((6, 32), device="cuda")
    Y = Y0.clone()
    w12.LoRA(A, B, scale).run(X, Y, to_dev_i32([0, 1, 0, 1, 0, -1]))
    _check(X, Y0, Y, A, B, scale, [0, 1, 0, 1, 0, -1])
    X[2, 3], X[3, 5] = float("inf"), float("nan")
    Z = Y0.clone()
    w12.LoRA(A, B, scale).run(X, Z, to_dev_i32([0, 1, 0, 1, 0, -1]))
    assert not torch.isfinite(Z[2]).any() and torch.isnan(Z[3]).all()
    assert torch.equal(Z[[0, 1, 4, 5]], Y[[0, 1, 4, 5]])


def test_beside_the_packed_projection():
    """Adapters on the rows of a W12 product, as a layer runs them."""
    from gpu_util import to_dev_bf16
    from oracle import w12_oracle as WO
    from speculative_decoding_verification_w12_gb300 import synthetic as S
    Wb, Xb = S.weights_bf16(256, 384, seed=2), S.activations_bf16(24, 384)
    A, B, scale, g = _make(4, 256, 384, 16)
    X = to_dev_bf16(Xb)
    ids = [0, 0, 1, -1, 3, 2] * 4
    Y = w12.gemm(X, w12.pack(to_dev_bf16(Wb)))
    base = Y.clone()
    w12.LoRA(A, B, scale).run(X, Y, to_dev_i32(ids))
    _check(X, base, Y, A, B, scale, ids)
    assert np.linalg.norm(base.cpu().numpy() - WO.gemm(Xb, WO.pack(Wb))) <= 1e-3 * np.linalg.norm(base.cpu().numpy())


@pytest.mark.parametrize("r", [8, 16, 24, 40, 104])
def test_an_infinity_of_a_row_meets_the_rank_alone(r):
    """Weights above zero: the row's outputs are infinite, not NaN (2 and 40 rows: both groupings)."""
    A, B, scale, g = _make(2, 48, 64, r)
    A, B = A.abs() + 0.01, B.abs() + 0.01
    for M in (2, 40):
        X, Y0 = torch.rand((M, 64), generator=g, device="cuda").bfloat16(), torch.zeros((M, 48), device="cuda")
        X[M // 2, 5] = float("inf")
        Y, ids = Y0.clone(), [m % 2 for m in range(M)]
        w12.LoRA(A, B, scale).run(X, Y, to_dev_i32(ids))
        assert (Y[M // 2] == float("inf")).all()
        Y[M // 2] = 0
        ids[M // 2] = -1
        _check(X, Y0, Y, A, B, scale, ids)


def test_sizes_past_32_bits():
    """Rows and adapters behind more than 2^31 values: bitwise what they give by themselves."""
    g = torch.Generator(device="cuda").manual_seed(4)
    scale = torch.ones(3, device="cuda")
    for K, N in ((2 ** 23, 32), (64, 2 ** 23)):
        A, B = (torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16) for s in ((3, 128, K), (3, N, 128)))
        X, Y = torch.randn((5, K), generator=g, device="cuda").bfloat16(), torch.zeros((5, N), device="cuda")
        alone = Y.clone()
        w12.LoRA(A, B, scale).run(X, Y, to_dev_i32([2] * 5))
        w12.LoRA(A[2:], B[2:], scale[2:]).run(X, alone, to_dev_i32([0] * 5))
        assert Y.abs().min() > 0 and torch.equal(Y, alone)
        del A, B, X, Y, alone
    M, apart = 200, 2 ** 24
    A, B, scale, g = _make(2, 64, 72, 16)
    X = torch.empty(M * apart, dtype=torch.bfloat16, device="cuda").as_strided((M, 72), (apart, 1))
    Y = torch.empty(M * apart, device="cuda").as_strided((M, 64), (apart, 1))
    X.copy_(torch.randn((M, 72), generator=g, device="cuda"))
    Y.zero_()
    ids = [m % 3 - 1 for m in range(M)]
    w12.LoRA(A, B, scale).run(X, Y, to_dev_i32(ids))
    _check(X, torch.zeros((M, 64), device="cuda"), Y, A, B, scale, ids)


def test_two_adapters_at_the_same_time():
    """Objects of their own (each has a workspace) on two streams."""
    sets = [_make(5, 512, 1024, r, seed=r) for r in (16, 64)]
    work = []
    for A, B, scale, g in sets:
        X, ids = torch.randn((64, 1024), generator=g, device="cuda").bfloat16(), to_dev_i32(np.arange(64) % 5)
        work.append((w12.LoRA(A, B, scale), X, ids, torch.cuda.Stream()))
    want = [lora.run(X, torch.zeros((64, 512), device="cuda"), ids) for lora, X, ids, _ in work]
    ys = [[torch.zeros((64, 512), device="cuda") for _ in range(20)] for _ in work]
    torch.cuda.synchronize()
    for i in range(20):
        for (lora, X, ids, s), y in zip(work, ys):
            lora.run(X, y[i], ids, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for some, w in zip(ys, want) for y in some)


@pytest.mark.parametrize("M,N,K,r", [(256, 80, 2072, 16), (200, 64, 520, 8), (129, 208, 1000, 64), (60, 16, 4104, 128), (31, 112, 5000, 32)])
def test_a_request_a_row_each_with_an_adapter_of_its_own(M, N, K, r):
    """More tiles than the clusters that the GPU holds, warps that go over several tiles; a row gets the
    same whatever the order of the rows."""
    A, B, scale, g = _make(M, N, K, r, seed=M)
    X, Y0 = torch.randn((M, K), generator=g, device="cuda").bfloat16(), torch.randn((M, N), generator=g, device="cuda")
    lora = w12.LoRA(A, B, scale)
    order = torch.randperm(M, generator=g, device="cuda")
    Y, Z = Y0.clone(), Y0[order].contiguous()
    lora.run(X, Y, torch.arange(M, dtype=torch.int32, device="cuda"))
    _check(X, Y0, Y, A, B, scale, list(range(M)))
    lora.run(X[order].contiguous(), Z, order.to(torch.int32))
    assert torch.equal(Z, Y[order])
