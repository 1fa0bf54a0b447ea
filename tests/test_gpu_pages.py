"""GPU page tables (w12_pages_update) against the list-based oracle: exact."""
import numpy as np
import pytest
import torch

from gpu_util import new_status, status_value, to_dev_i32
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu
w12 = pytest.importorskip("speculative_decoding_verification_w12_gb300.w12")


def _pt(table, used, free, n_free, P):
    return w12.PageTable(to_dev_i32(table), to_dev_i32(used), to_dev_i32(free), to_dev_i32([n_free]), P)


def _state(pt):
    return (pt.table.cpu().tolist(), pt.used.cpu().tolist(), pt.free.cpu().tolist(), int(pt.n_free.item()))


def _start_state(B, max_pages, n_pages, g):
    ids = g.permutation(n_pages).tolist()
    table, used = [], []
    for b in range(B):
        n = int(g.integers(0, max_pages // 2 + 1))
        n = min(n, len(ids))
        table.append(ids[:n] + [-1] * (max_pages - n))
        used.append(n)
        ids = ids[n:]
    return table, used, ids + [0] * (n_pages - len(ids)), len(ids)


@pytest.mark.parametrize("B,max_pages,P,T", [(1, 4, 16, 1), (3, 9, 32, 70), (33, 6, 64, 16), (600, 12, 128, 5), (1300, 3, 16, 33),
                                             (2, 700, 16, 9000)])
def test_random_steps_match_the_oracle(B, max_pages, P, T):
    g = np.random.default_rng(B + T)
    n_pages = B * max_pages
    table, used, free, n_free = _start_state(B, max_pages, n_pages, g)
    pt = _pt(table, used, free, n_free, P)
    for step in range(6):
        most = max_pages * P
        start = g.integers(0, most + 1, B)
        add = np.minimum(g.integers(0, T + 1, B), most - start)
        reserve = step % 3 != 2
        want = O.pages_update(table, used, free, n_free, start.tolist(), add.tolist() if reserve else None,
                              T if reserve else 0, P)
        st = new_status()
        if reserve:
            slots = pt.reserve(to_dev_i32(start), to_dev_i32(add), T, status=st)
            assert slots.cpu().tolist() == want[4]
        else:
            pt.trim(to_dev_i32(start), status=st)
        code = status_value(st)
        assert (code in want[5]) if want[5] else code == 0
        table, used, free, n_free = want[:4]
        got = _state(pt)
        assert got[0] == table and got[1] == used and got[3] == n_free
        assert got[2][:n_free] == free[:n_free]


def test_reserve_then_trim_restores_everything():
    B, P, T = 16, 64, 64
    g = np.random.default_rng(3)
    table, used, free, n_free = _start_state(B, 20, 400, g)
    start = [u * P - int(g.integers(0, P)) if u else 0 for u in used]
    pt = _pt(table, used, free, n_free, P)
    before = _state(pt)
    pt.reserve(to_dev_i32(start), to_dev_i32([T] * B), T)
    assert _state(pt) != before
    pt.trim(to_dev_i32(start))
    assert _state(pt) == before


def test_shortage_serves_in_order():
    # Request 0 fits, 1 does not, 2 would but comes later, 3 needs nothing, 4 shrinks.
    table = [[-1] * 4, [-1] * 4, [-1] * 4, [0, -1, -1, -1], [1, 2, 3, -1]]
    args = ([0, 0, 0, 3, 1], [20, 40, 1, 5, 0])
    st = new_status()
    pt = _pt(table, [0, 0, 0, 1, 3], [9, 8, 7, 4, 5, 6], 3, 16)
    slots = pt.reserve(to_dev_i32(args[0]), to_dev_i32(args[1]), 40, status=st)
    want = O.pages_update(table, [0, 0, 0, 1, 3], [9, 8, 7, 4, 5, 6], 3, *args, 40, 16)
    assert status_value(st) == 3 == O.ERR_WORKSPACE
    assert slots.cpu().tolist() == want[4] and _state(pt)[0] == want[0] and _state(pt)[1] == want[1]
    assert _state(pt)[3] == want[3] == 3 and _state(pt)[2][:3] == want[2][:3]


@pytest.mark.parametrize("start,add,used", [([-1, 0], [1, 1], [0, 0]), ([0, 0], [-2, 1], [0, 0]), ([0, 0], [5, 1], [0, 0]),
                                            ([60, 0], [5, 1], [0, 0]), ([0, 0], [1, 1], [5, 0]), ([0, 0], [1, 1], [-1, 0])])
def test_bad_lengths_leave_the_request_as_it_is(start, add, used):
    st = new_status()
    pt = _pt([[0, 1, 2, 3], [-1] * 4], used, [7, 6, 5, 4], 4, 16)
    slots = pt.reserve(to_dev_i32(start), to_dev_i32(add), 4, status=st)
    assert status_value(st) == 1
    assert slots.cpu().tolist() == [[-1] * 4, [4 * 16, -1, -1, -1]]
    assert _state(pt) == ([[0, 1, 2, 3], [4, -1, -1, -1]], [used[0], 1], [7, 6, 5, 4], 3)


def test_bad_free_count_is_flagged():
    st = new_status()
    pt = _pt([[-1, -1]], [0], [3, 2, 1], 9, 16)
    pt.reserve(to_dev_i32([0]), to_dev_i32([1]), 1, status=st)
    assert status_value(st) == 1


def test_most_requests_of_a_call():
    B, P = 8192, 16
    pt = w12.PageTable.create(B, 2, 2 * B, P)
    new = torch.arange(B, dtype=torch.int32, device="cuda") % 33
    slots = pt.reserve(torch.zeros(B, dtype=torch.int32, device="cuda"), new, 32)
    want = O.pages_update([[-1, -1]] * B, [0] * B, list(range(2 * B - 1, -1, -1)), 2 * B, [0] * B, new.tolist(), 32, P)
    assert slots.cpu().tolist() == want[4] and pt.table.cpu().tolist() == want[0]


def test_another_stream_and_a_graph():
    B, P, T = 4, 16, 20
    pt = w12.PageTable.create(B, 8, 32, P)
    start, new = to_dev_i32([0, 3, 16, 17]), to_dev_i32([20, 1, 0, 7])
    want = O.pages_update([[-1] * 8] * B, [0] * B, list(range(31, -1, -1)), 32, start.tolist(), new.tolist(), T, P)[4]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = pt.reserve(start, new, T, stream=s)
    pt.trim(to_dev_i32([0] * B), stream=s)
    s.synchronize()
    assert a.cpu().tolist() == want
    zero, out = to_dev_i32([0] * B), torch.empty((B, T), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pt.reserve(start, new, T, slots=out)
        pt.trim(zero)
    for _ in range(3):
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert out.cpu().tolist() == want


def test_binding_refusals():
    pt = w12.PageTable.create(2, 4, 8, 16)
    i = to_dev_i32([0, 0])
    with pytest.raises(ValueError):
        pt.reserve(i.long(), i, 4)
    with pytest.raises(ValueError):
        pt.reserve(to_dev_i32([0]), i, 4)
    with pytest.raises(ValueError):
        pt.reserve(i, i, 4, slots=torch.empty((2, 5), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        w12.PageTable(pt.table.cpu(), pt.used, pt.free, pt.n_free, 16)
    bad = w12.PageTable.create(2, 4, 8, 24)
    with pytest.raises(w12.W12Error) as e:
        bad.reserve(i, i, 4)
    assert e.value.code == 2


def test_positions_past_2_to_the_31():
    """A request that grows over position 2^31: slots of its last held page, then of the page it takes."""
    held, P = 1 << 24, 128
    table = torch.zeros((1, held + 2), dtype=torch.int32, device="cuda")
    pages = w12.PageTable(table, to_dev_i32([held]), to_dev_i32([1, 0]), to_dev_i32([1]), P)
    st = new_status()
    slots = pages.reserve(to_dev_i32([2 ** 31 - 4]), to_dev_i32([8]), 9, status=st)
    assert status_value(st) == 0
    assert slots.tolist() == [[124, 125, 126, 127, 128, 129, 130, 131, -1]]
    assert pages.used.item() == held + 1 and pages.n_free.item() == 0 and table[0, held].item() == 1
