"""Rotation, rotated appends, tree positions, prompt attention and adapters without a GPU: arguments
that the binding and the C ABI refuse, memory on the call's stream, and what the sources of the prompt
kernel have to hold (copies waited for, registers)."""
import ctypes
import os
import re

import pytest
import torch

from speculative_decoding_verification_w12_gb300 import build as B
from speculative_decoding_verification_w12_gb300 import w12
from test_refusals_cpu import calls, i32  # noqa: F401
from test_streams_cpu import Cuda, Stream, cuda, record  # noqa: F401

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rope(d=64, rot=64, n=32, **kw):
    return w12.Rope(cuda(n, rot), d, **kw)


def _cache(Hkv=2, d=64, P=16):
    return w12.KV4Cache(cuda(4, Hkv, P * (d + 8), dtype=torch.uint8), P, d)


def _lora(n=3, r=16, K=64, N=32):
    return w12.LoRA(cuda(n, r, K, dtype=BF16), cuda(n, N, r, dtype=BF16), cuda(n))


def refused(*errors):
    return pytest.raises(errors or (ValueError, TypeError))


def test_rope_refuses(calls):  # noqa: F811
    for bad in (dict(rot=24), dict(rot=0), dict(rot=128), dict(d=96, rot=64), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(q_norm=cuda(63)), dict(k_norm=cuda(64, dtype=BF16)), dict(q_norm=torch.ones(64))):
        with refused():
            _rope(**bad)
    with refused():
        w12.Rope(cuda(32, 128)[:, :64], 64)
    r = _rope()
    Q, K, pos = cuda(5, 3, 64), cuda(5, 2, 64), i32(5)
    r.run(Q, K, pos)
    for q, k, p in ((Q, cuda(4, 2, 64), pos), (Q, K, i32(4)), (Q, cuda(5, 2, 64, dtype=BF16), pos), (cuda(5, 3, 128), K, pos), (None, None, pos),
                    (Q, K, cuda(5, dtype=torch.int64)), (torch.ones(5, 3, 64), K, pos), (cuda(5, 64), K, pos), (cuda(5, 3, 64, dtype=torch.float64), K, pos),
                    (cuda(5, 64, 3).transpose(1, 2), K, pos)):
        with refused():
            r.run(q, k, p)
    with refused():
        r.run(Q, K, pos, dtype=torch.float64)
    with refused():
        r.run(Q, K, pos, out=(cuda(5, 3, 64), cuda(5, 2, 64)))          # of another type than bf16
    with refused():
        r.run(Q, K, pos, out=(cuda(5, 3, 64, dtype=BF16), cuda(5, 2, 65, dtype=BF16)))
    assert calls == ["w12_qk_norm_rope"]
    r.run(Q[:0], K[:0], pos[:0])
    assert calls == ["w12_qk_norm_rope"]                                # nothing to do


def test_append_rope_refuses(calls):  # noqa: F811
    c, r = _cache(), _rope()
    K, V, Q, slots, pos = cuda(5, 2, 64), cuda(5, 2, 64), cuda(5, 6, 64), i32(5), i32(5)
    assert c.append_rope(K, V, slots, r, pos) is None
    assert c.append_rope(K, V, slots, r, pos, Q=Q).dtype is BF16
    n = len(calls)
    for kw in (dict(V=cuda(5, 2, 64, dtype=BF16)), dict(V=cuda(4, 2, 64)), dict(K=cuda(5, 3, 64), V=cuda(5, 3, 64)), dict(slots=i32(4)),
               dict(slots=cuda(5, dtype=torch.int64)), dict(positions=i32(6)), dict(rope=_rope(128, 128)), dict(Q=cuda(4, 6, 64)),
               dict(Q=cuda(5, 6, 64, dtype=F16)), dict(Q=cuda(5, 6, 128)), dict(out=cuda(5, 6, 64, dtype=BF16)), dict(Q=Q, out=cuda(5, 6, 64))):
        a = dict(K=K, V=V, slots=slots, rope=r, positions=pos) | kw
        with refused():
            c.append_rope(**a)
    assert len(calls) == n


def test_tree_positions_refuses(calls):  # noqa: F811
    w12.tree_positions(i32(3), i32(3, 4))
    w12.tree_positions(i32(3), T=7, q_len=i32(3))
    for bad in (dict(parents=i32(2, 4)), dict(), dict(parents=i32(3, 4), T=5), dict(T=4, q_len=i32(2)), dict(T=4, out=i32(3, 5)),
                dict(parents=cuda(3, 4, dtype=torch.int64))):
        with refused():
            w12.tree_positions(i32(3), **bad)
    assert calls == ["w12_tree_positions"] * 2


def test_prompt_attention_refuses(calls):  # noqa: F811
    def qkv(n=6, Hq=4, Hkv=2, d=64, dtype=BF16):
        return dict(Q=cuda(n, Hq, d, dtype=dtype), K=cuda(n, Hkv, d, dtype=dtype), V=cuda(n, Hkv, d, dtype=dtype), cu_seqlens=i32(3))
    w12.prompt_attention(**qkv())
    for bad in (dict(K=cuda(5, 2, 64, dtype=BF16)), dict(V=cuda(6, 1, 64, dtype=BF16)), dict(V=cuda(6, 2, 64, dtype=F16)), dict(Q=cuda(6, 4, 64)),
                dict(Q=cuda(6, 4, 128, dtype=BF16)), dict(cu_seqlens=cuda(3, dtype=torch.int64)), dict(cu_seqlens=i32(1, 3)), dict(cu_seqlens=i32(0)),
                dict(out=cuda(6, 4, 64, dtype=F16)), dict(out=cuda(6, 4, 65, dtype=BF16))):
        with refused():
            w12.prompt_attention(**(qkv() | bad))
    assert calls == ["w12_prompt_attention"]


def test_lora_refuses(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    lora = _lora()
    X, Y, ids = cuda(5, 64, dtype=BF16), cuda(5, 32), i32(5)
    assert lora.run(X, Y, ids) is Y
    n = len(calls)
    for bad in ((cuda(5, 63, dtype=BF16), Y, ids), (cuda(5, 64), Y, ids), (X, cuda(5, 32, dtype=BF16), ids), (X, cuda(4, 32), ids), (X, Y, i32(4)),
                (X, cuda(32, 5).t(), ids), (cuda(257, 64, dtype=BF16), cuda(257, 32), i32(257))):
        with refused():
            lora.run(*bad)
    assert len(calls) == n
    for bad in ((cuda(3, 16, 64, dtype=BF16), cuda(3, 32, 8, dtype=BF16), cuda(3)), (cuda(3, 16, 64), cuda(3, 32, 16, dtype=BF16), cuda(3)),
                (cuda(3, 12, 64, dtype=BF16), cuda(3, 32, 12, dtype=BF16), cuda(3)), (cuda(3, 136, 64, dtype=BF16), cuda(3, 32, 136, dtype=BF16), cuda(3)),
                (cuda(3, 16, 60, dtype=BF16), cuda(3, 32, 16, dtype=BF16), cuda(3)), (cuda(3, 16, 64, dtype=BF16), cuda(3, 24, 16, dtype=BF16), cuda(3)),
                (cuda(3, 16, 64, dtype=BF16), cuda(3, 32, 16, dtype=BF16), cuda(2)), (cuda(16, 64, dtype=BF16), cuda(3, 32, 16, dtype=BF16), cuda(3))):
        with refused():
            w12.LoRA(*bad)


CALLS = {
    "rope": lambda s: _rope().run(cuda(5, 3, 64), cuda(5, 2, 64), i32(5), stream=s),
    "append_rope": lambda s: _cache().append_rope(cuda(5, 2, 64), cuda(5, 2, 64), i32(5), _rope(), i32(5), Q=cuda(5, 6, 64), stream=s),
    "tree_positions": lambda s: w12.tree_positions(i32(3), i32(3, 4), stream=s),
    "prompt_attention": lambda s: w12.prompt_attention(*(cuda(6, h, 64, dtype=BF16) for h in (4, 2, 2)), i32(2), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_belongs_to_the_calls_stream(record, name):  # noqa: F811
    made, launched = record
    CALLS[name](Stream())
    assert made and all(on for _, on in made), made
    assert launched and all(stream == 5 for _, stream in launched)


# ---------------------------------------------------------------- the C ABI, on the host
@pytest.fixture(scope="module")
def L():
    B.build()
    return w12.lib()


@pytest.fixture(scope="module")
def at():
    buf = (ctypes.c_uint8 * 8192)()
    at.buf = buf
    return (ctypes.addressof(buf) + 63) // 64 * 64


OK = 0 if torch.cuda.is_available() else 8


def test_c_rope(L, at):
    def call(dtype=1, n=0, Q=at, K=at, q=at, k=at, out=1, d=128, Hq=4, Hkv=2, pos=at, **kw):
        r = w12._Rope(*(kw.get(f, v) for f, v in (("table", at), ("max_pos", 8), ("rot", 128), ("pairs", 0), ("qn", at), ("kn", None), ("eps", 1e-6))))
        return L.w12_qk_norm_rope(ctypes.byref(r), d, Q, 512, 128, Hq, K, 256, 128, Hkv, dtype, n, pos, q, k, out, None, None)
    assert call() == OK and call(Q=None, q=None) == OK and call(K=None, k=None) == OK and call(d=64, rot=16) == OK
    for bad in (dict(dtype=3), dict(n=-1), dict(Q=None, K=None), dict(q=None), dict(q=at + 8), dict(k=at + 4), dict(out=-1), dict(pos=None), dict(table=None),
                dict(table=at + 8), dict(qn=at + 4), dict(eps=0.0), dict(eps=float("nan")), dict(Q=at + 1)):
        assert call(**bad) == 1, bad
    for bad in (dict(d=96), dict(rot=24), dict(rot=0), dict(rot=144), dict(max_pos=0), dict(max_pos=2 ** 31), dict(Hq=0), dict(Hkv=1025), dict(n=2 ** 31 - 1)):
        assert call(**bad) == 2, bad
    assert call(eps=0.0, qn=None) == OK                                   # no norm: eps is not looked at


def test_c_append_rope(L, at):
    def call(n=0, Q=at, K=at, V=at, q=at, slots=at, pos=at, pool=at, P=16, d=64, dtype=0):
        c, r = w12._KV4(pool, 4, 2, d, P), w12._Rope(at, 8, 64, 0, None, None, 0)
        return L.w12_kv4_append_rope(ctypes.byref(c), ctypes.byref(r), Q, 256, 64, 4, K, 128, 64, V, 128, 64, dtype, n, pos, slots, q, None, None)
    assert call() == OK and call(Q=None, q=None) == OK
    for bad in (dict(K=None), dict(V=None), dict(q=None), dict(slots=None), dict(pos=None), dict(pool=None), dict(pool=at + 8), dict(q=at + 8), dict(dtype=5),
                dict(K=at + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(P=17), dict(d=80), dict(n=2 ** 31 - 1)):
        assert call(**bad) == 2, bad


def test_c_tree_positions(L, at):
    f = L.w12_tree_positions
    assert f(None, at, at, 1, 4, at, None, None) == 1 and f(at, at, at, 1, 4, None, None, None) == 1
    for b, t, parents in ((0, 4, at), (1, 0, at), (1, 257, at), (65536, 4, None)):
        assert f(at, parents, None, b, t, at, None, None) == 2


def test_c_prompt_attention(L, at):
    def call(Q=at, qt=256, qh=64, K=at, kt=128, kh=64, V=at, vt=128, vh=64, dtype=1, total=0, cu=at, b=1, Hq=4, Hkv=2, d=64, scale=0.1, O=at):
        return L.w12_prompt_attention(Q, qt, qh, K, kt, kh, V, vt, vh, dtype, total, cu, b, Hq, Hkv, d, scale, O, None, None)
    assert call() == OK and call(b=0, total=4) == OK                      # nothing to do
    for bad in (dict(dtype=0), dict(dtype=3), dict(cu=None), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(total=4, Q=None),
                dict(total=4, O=at + 16), dict(total=4, K=at + 8), dict(total=4, qt=0), dict(total=4, kh=-64), dict(total=4, vt=100)):
        assert call(**bad) == 1, bad
    for bad in (dict(b=-1), dict(total=-1), dict(total=2 ** 31), dict(Hkv=0), dict(Hq=5), dict(Hq=258), dict(d=96), dict(b=65536)):
        assert call(**bad) == 2, bad


def test_c_lora(L, at):
    def call(X=at, xs=64, M=2, Y=at, ys=32, ids=at, ws=at, size=8192, A=at, Bm=at, scale=at, N=32, K=64, n=2, r=16):
        a = w12._Adapters(A, Bm, scale, N, K, n, r)
        return L.w12_lora(X, xs, M, ctypes.byref(a), ids, Y, ys, ws, size, None, None)
    for bad in (dict(X=None), dict(Y=None), dict(ids=None), dict(A=None), dict(Bm=None), dict(scale=None), dict(X=at + 8), dict(Y=at + 4), dict(A=at + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(M=0), dict(M=257), dict(r=12), dict(r=136), dict(r=0), dict(N=24), dict(K=60), dict(n=0), dict(xs=56), dict(xs=68), dict(ys=34), dict(ys=16)):
        assert call(**bad) == 2, bad
    for bad in (dict(ws=None), dict(size=100), dict(ws=at + 8)):
        assert call(**bad) == 3, bad
    assert L.w12_lora_ws_bytes(256, 64, 64) > L.w12_lora_ws_bytes(16, 64, 64) > 0 == L.w12_lora_ws_bytes(257, 64, 64)


# ---------------------------------------------------------------- the prompt kernel's source
def test_prompt_kernel_waits_for_its_copies_and_shares_its_registers():
    src = open(os.path.join(B.CSRC, "w12_prompt.cu")).read()
    kernel = src[src.index("__global__"):]
    tail = kernel[kernel.rindex("\n  cta_sync();"):]
    for bar in ("full", "q_full"):
        assert re.search(r"mbar_wait\(&" + bar + r"\[[^;]*drain_limit_ns", tail), bar
    assert not re.search(r"(?<!mbar_)\bwait(_all)?\(", tail[:tail.index("tmem_dealloc")])
    regs = dict(re.findall(r"(k\w+Regs) = (\d+)", src))
    threads = int(re.search(r"kThreads = (\d+)", src).group(1))
    assert 8 * int(regs["kSoftRegs"]) + (threads // 32 - 8) * int(regs["kRestRegs"]) <= threads // 32 * int(regs["kLaunchRegs"])
    assert int(regs["kLaunchRegs"]) * threads <= 65536 and all(int(v) % 8 == 0 for v in regs.values())
    calls_ = re.findall(r"(?:fewer|more)_registers<(\w+)>\(\)", kernel)
    assert sorted(calls_) == ["kRestRegs", "kSoftRegs"]                   # one instruction a warpgroup


class Elsewhere(Cuda):
    """Passes for a tensor of device 1."""
    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(w12, "_device_index", lambda: 0)
    other = lambda *s, dtype=F32: cuda(*s, dtype=dtype).as_subclass(Elsewhere)  # noqa: E731
    r, c, lora = _rope(), _cache(), _lora()
    n = len(calls)
    for call in (lambda f: r.run(f(5, 3, 64), cuda(5, 2, 64), i32(5)), lambda f: r.run(cuda(5, 3, 64), f(5, 2, 64), i32(5)),
                 lambda f: c.append_rope(f(5, 2, 64), cuda(5, 2, 64), i32(5), r, i32(5)),
                 lambda f: w12.tree_positions(f(3, dtype=torch.int32), T=4),
                 lambda f: w12.prompt_attention(f(6, 4, 64, dtype=BF16), cuda(6, 2, 64, dtype=BF16), cuda(6, 2, 64, dtype=BF16), i32(2)),
                 lambda f: lora.run(f(5, 64, dtype=BF16), cuda(5, 32), i32(5))):
        with refused(ValueError):
            call(other)
        assert len(calls) == n
        call(cuda)
        n += 1
        assert len(calls) == n
    monkeypatch.setattr(w12, "_device_index", lambda: 1)
    r.run(other(5, 3, 64), None, i32(5))                                  # the current one


def test_c_longest_chunk(L, at):
    f = L.w12_tree_positions
    assert f(at, None, None, 1, 2 ** 23 + 1, at, None, None) == 2 and f(at, None, None, 1, 2 ** 31 - 1, at, None, None) == 2
