"""Measured cases of what a layer does between its products: rotation, cache writes, prompt attention, adapters.

Four groups of operators, as a serving program uses them around the products of a layer:

  rope     norms of queries and keys for each head and the rotation by position, in one pass;
  append   the same on the way into the paged 4-bit cache: keys are normed, rotated and
           quantised, values quantised, queries of the same rows rotated beside them; for draft
           trees the positions come from the tree. The written rows are read back;
  prompt   causal attention over whole prompts, packed one behind the other, grouped heads;
  lora     low-rank adapters of many requests, added to the rows of a shared projection.

``run`` computes the plain form (torch, fp32) unless ``own`` is set; then it makes the calls
of the framework's w12 binding. Both work on the same buffers.

Rotation: the table is fp32 [positions, rot], the cosines of a position's rot / 2 angles and then
their sines. Values i and i + rot/2 of a head are a pair, or with interleaved pairs 2i and 2i + 1;
those past rot stay. A norm is x / sqrt(mean x^2 + eps) times the head's weights, its factor
rounded once to fp32. A position of -1 is a row without a token: it reads as zero.

The cache is that of the library ("KV4"): a pool uint8 [n_pages, Hkv, P (d + 8)]; per kv head K
codes [P, d/2], V codes, K parameters [P, 2], V parameters (bf16 scale s, bf16 centre z); a row
stores x as z + s (q - 8), q in 0..15. Word w of a row's codes holds dims 8w..8w+7: nibble j
(j < 4) is dim 8w + 2j, nibble j + 4 is dim 8w + 2j + 1; with d = 128 the row's two 32-byte halves
are swapped in rows whose index in the page has bit 1 set. Slot = page P + row.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The drafted block of one request, straight from the fp32 output of the qkv product (views of it).
        dict(name="rope-block-16-f32", op="rope", n=16, Hq=40, Hkv=8, d=128, rot=128, pairs=False, norm=True, dtype="float32", out="bfloat16", strided=True, max_pos=32768),
        # Prompt rows of a layer: queries and keys for the attention over them.
        dict(name="rope-prompt-16384", op="rope", n=16384, Hq=40, Hkv=8, d=128, rot=128, pairs=False, norm=True, dtype="bfloat16", out="bfloat16", strided=True, max_pos=32768),
        # Draft trees of four requests: positions from the trees, queries rotated, keys and values cached.
        dict(name="append-tree-4x64-f32", op="append", B=4, T=64, Hq=40, Hkv=8, d=128, rot=128, page=64, pairs=False, norm=True, dtype="float32", tree=True, strided=True, len_max=8192),
        # Single tokens of a batch, small heads rotated in part and by neighbours, some requests idle.
        dict(name="append-decode-64-d64", op="append", B=64, T=1, Hq=10, Hkv=2, d=64, rot=32, page=16, pairs=True, norm=False, dtype="bfloat16", tree=False, strided=False, len_max=8192),
        # Prompts of up to 8192 tokens into the cache (their queries are rotated elsewhere).
        dict(name="append-prompt-4x8192", op="append", B=4, T=8192, Hq=0, Hkv=8, d=128, rot=128, page=64, pairs=False, norm=True, dtype="bfloat16", tree=False, strided=False, len_max=0),
        # One prompt of an odd length.
        dict(name="prompt-1x777", op="prompt", B=1, len_max=777, Hq=40, Hkv=8, d=128, dtype="bfloat16", strided=False),
        # A batch of short prompts of all lengths, none and one token among them.
        dict(name="prompt-64x300", op="prompt", B=64, len_max=300, Hq=40, Hkv=8, d=128, dtype="bfloat16", strided=True),
        # Four long prompts, ragged, as views of the qkv product's rows.
        dict(name="prompt-4x4096", op="prompt", B=4, len_max=4096, Hq=40, Hkv=8, d=128, dtype="bfloat16", strided=True),
        # One long prompt in fp16 with 64-wide heads.
        dict(name="prompt-1x8192-f16-d64", op="prompt", B=1, len_max=8192, Hq=32, Hkv=8, d=64, dtype="float16", strided=False),
        # The drafted block of one request beside the attention's output projection.
        dict(name="lora-1x16-o", op="lora", M=16, N=5120, K=5120, r=16, adapters=8, used=1, idle=False),
        # Single tokens of 64 requests, each with an adapter of its own or none, beside the qkv product.
        dict(name="lora-64x1-qkv", op="lora", M=64, N=7168, K=5120, r=16, adapters=128, used=48, idle=True),
        # Drafted blocks of 16 requests with adapters of a higher rank beside gate and up.
        dict(name="lora-16x16-gate-up", op="lora", M=256, N=34816, K=5120, r=64, adapters=32, used=16, idle=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(40, 8), (32, 8), (16, 2), (8, 8), (10, 2), (12, 4), (16, 1)]


def draw(rng):
    op = rng.choice(["rope", "append", "append", "prompt", "prompt", "lora"])
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice([64, 128])
    turn = dict(rot=rng.choice([d, d, d // 2, d // 4]), pairs=rng.random() < 0.3, norm=rng.random() < 0.7)
    kinds = ["float32", "bfloat16", "float16"]
    if op == "rope":
        c = dict(op=op, n=_logint(rng, 1, 16384), Hq=Hq, Hkv=Hkv, d=d, **turn, dtype=rng.choice(kinds), out=rng.choice(kinds), strided=rng.random() < 0.5, max_pos=_logint(rng, 16, 65536))
        return _within(c, "n")
    if op == "append":
        c = dict(op=op, Hkv=Hkv, d=d, **turn, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(kinds), strided=rng.random() < 0.5)
        if rng.random() < 0.7:
            c.update(B=_logint(rng, 1, 16), T=_logint(rng, 1, 64), Hq=Hq, tree=rng.random() < 0.5, len_max=_logint(rng, 16, 32768))
        else:
            c.update(B=rng.randint(1, 4), T=_logint(rng, 65, 8191), Hq=rng.choice([0, Hq]), tree=False, len_max=0)
        return _within(c, "T")
    if op == "prompt":
        return _within(dict(op=op, B=_logint(rng, 1, 64), len_max=_logint(rng, 1, 8192), Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bfloat16", "float16"]), strided=rng.random() < 0.5), "len_max")
    M = _logint(rng, 1, 256)
    c = dict(op=op, M=M, N=rng.choice([5120, 7168, 16 * _logint(rng, 1, 2176)]), K=rng.choice([5120, 17408, 8 * _logint(rng, 1, 2176)]), r=rng.choice([8, 16, 24, 32, 64, 128]),
             adapters=_logint(rng, 1, 128), idle=rng.random() < 0.5)
    c["used"] = _logint(rng, 1, min(M, c["adapters"]))
    return _within(c, "N", 16)


def _within(c, size, unit=1):
    """The case with `size` cut until it costs no more than the largest listed case of its operator."""
    most = [work(x) for x in listed() if x["op"] == c["op"]]
    while c[size] > unit and any(work(c)[k] > max(w[k] for w in most) for k in ("bytes", "flops")) or _scores(c) > 4 * 40 * 4096 * 4096:
        c[size] = max(1, c[size] // unit * 2 // 3) * unit
    return c


def _scores(c):
    """Scores of a padded batch of prompts."""
    return c["B"] * c["Hq"] * c["len_max"] ** 2 if c["op"] == "prompt" else 0


def _lengths(c):
    """(tokens already cached, new tokens) of each request: plain lists, from the case alone."""
    cached, new = [], []
    for b in range(c["B"]):
        f = ((b + 1) * 0.6180339887498949) % 1.0
        if c["op"] == "prompt":
            cached.append(0)
            new.append(c["len_max"] if b == 0 else 0 if b % 8 == 5 else 1 if b % 8 == 6 else c["len_max"] - int(f * c["len_max"] * 0.75))
        else:
            cached.append(int(f * c["len_max"]))
            new.append(0 if b % 16 == 7 else c["T"] - int(f * (c["T"] // 4)))
    return cached, new


def work(c):
    e = 4 if c.get("dtype") == "float32" else 2
    if c["op"] == "lora":
        rows = _adapter_rows(c)
        used, live = len(set(a for a in rows if a >= 0)), sum(a >= 0 for a in rows)
        return dict(bytes=2 * live * c["K"] + 2 * used * c["r"] * (c["K"] + c["N"]) + 8 * live * c["N"] + 4 * c["M"], flops=2 * live * c["r"] * (c["K"] + c["N"]))
    if c["op"] == "rope":
        rows = c["n"] * (c["Hq"] + c["Hkv"])
        out = 4 if c["out"] == "float32" else 2
        return dict(bytes=rows * c["d"] * (e + out) + 4 * min(c["n"], c["max_pos"]) * c["rot"] + 4 * c["n"], flops=rows * (4 * c["d"] + 3 * c["rot"]))
    cached, new = _lengths(c)
    if c["op"] == "append":
        kv, q = sum(new) * c["Hkv"], sum(new) * c["Hq"]
        lost = (c["B"] * c["T"] - sum(new)) * (c["Hq"] + 2 * c["Hkv"]) * c["d"] * 2  # rows without a token are written too
        return dict(bytes=kv * (2 * c["d"] * e + 2 * (c["d"] + 8) + 4 * c["d"]) + q * c["d"] * (e + 2) + lost + 4 * sum(new) * c["rot"],
                    flops=(kv + q) * (4 * c["d"] + 3 * c["rot"]) + 16 * kv * c["d"])
    pairs = sum(n * (n + 1) // 2 for n in new)
    return dict(bytes=2 * sum(new) * c["d"] * (2 * c["Hq"] + 2 * c["Hkv"]), flops=4 * pairs * c["Hq"] * c["d"])


def _adapter_rows(c):
    """The adapter of each row, -1 without one: rows of a request are neighbours."""
    spread = [(7 * k + 3) % c["adapters"] if math.gcd(7, c["adapters"]) == 1 else k for k in range(c["used"])]
    each = max(1, -(-c["M"] // c["used"]))
    rows = [spread[(m // each) % c["used"]] for m in range(c["M"])]
    return [-1 if c["idle"] and m % 4 == 1 else a for m, a in enumerate(rows)]


# ------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _inv_freq(rot):
    """Angle per position of each pair, in fp64."""
    return THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def _table(positions, rot):
    """Cosines and sines of every position's angles: worked out in fp64, kept in fp32."""
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * _inv_freq(rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rows(c, n, g):
    """Q, K and V rows [n, H, d] of one qkv product: views of its rows, or each on its own."""
    Hq, Hkv, d, t = c["Hq"], c["Hkv"], c["d"], getattr(torch, c["dtype"])
    wide = torch.randn((n, (Hq + 2 * Hkv) * d), generator=g, device="cuda").to(t)
    parts = [x.unflatten(1, (-1, d)) for x in wide.split([Hq * d, Hkv * d, Hkv * d], 1)] if Hq else [None] + [x.unflatten(1, (-1, d)) for x in wide.split([Hkv * d, Hkv * d], 1)]
    return parts if c["strided"] else [x if x is None else x.contiguous() for x in parts]


def _norms(c, g):
    """Weights of the norms of queries and keys."""
    if not c["norm"]:
        return None, None
    return tuple(1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda") for _ in range(2))


def prepare(c, seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "lora":
        n = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        M, N, K, rank = c["M"], c["N"], c["K"], c["r"]
        names = list(range(c["adapters"]))
        r.shuffle(names)
        s = dict(c=c, X=n(M, K).bfloat16(), Y=n(M, N), A=(n(c["adapters"], rank, K) * K ** -0.5).bfloat16(), B=(n(c["adapters"], N, rank) * rank ** -0.5).bfloat16())
        s["scale"] = 0.5 + torch.rand(c["adapters"], generator=g, device="cuda")
        s["ids"] = _i32([-1 if a < 0 else names[a] for a in _adapter_rows(c)])
        return s
    if c["op"] == "prompt":
        lens = _lengths(c)[1]
        cu = [sum(lens[:b]) for b in range(c["B"] + 1)]
        Q, K, V = _rows(c, cu[-1], g)
        return dict(c=c, Q=Q, K=K, V=V, cu=_i32(cu), longest=max(lens))
    if c["op"] == "rope":
        Q, K, _ = _rows(c, c["n"], g)
        qn, kn = _norms(c, g)
        at = torch.randint(0, c["max_pos"], (c["n"],), generator=g, device="cuda", dtype=torch.int32)
        return dict(c=c, Q=Q, K=K, positions=at, table=_table(c["max_pos"], c["rot"]), q_norm=qn, k_norm=kn)
    cached, new = _lengths(c)
    P, B, T = c["page"], c["B"], c["T"]
    need = [-(-(a + n) // P) for a, n in zip(cached, new)]
    pages = list(range(sum(-(-n // P) + 1 for n in new)))  # the pages that the new tokens touch, in any order
    r.shuffle(pages)
    slots, at = [], 0
    for a, n, k in zip(cached, new, need):
        first = a // P
        slots.append([pages[at + (a + i) // P - first] * P + (a + i) % P for i in range(n)] + [-1] * (T - n))
        at += max(0, k - first)
    Q, K, V = _rows(c, B * T, g)
    qn, kn = _norms(c, g)
    s = dict(c=c, Q=Q, K=K, V=V, slots=_i32(slots).flatten(), q_norm=qn, k_norm=kn, prefix=_i32(cached), new=_i32(new))
    s["pool"] = torch.zeros((len(pages), c["Hkv"], P * (c["d"] + 8)), dtype=torch.uint8, device="cuda")
    s["table"] = _table(max(a + n for a, n in zip(cached, new)) + 1, c["rot"])
    if c["tree"]:
        s["parents"] = _i32([[-1] + [r.randrange(i) if r.random() < 0.7 else i - 1 for i in range(1, T)] for _ in range(B)])
    else:
        i = torch.arange(T, dtype=torch.int32, device="cuda")[None]
        s["positions"] = torch.where(i < s["new"][:, None], s["prefix"][:, None] + i, -1)
    return s


# ------------------------------------------------------------------ plain forms
def _turned(x, weight, positions, s):
    """Rows [n, H, d] normed (where there is a weight) and rotated, in fp32."""
    c = s["c"]
    x = x.float()
    if weight is not None:
        mean = x.double().square().mean(-1, keepdim=True)
        x = x * (mean + torch.tensor(EPS, dtype=torch.float32, device="cuda").double()).rsqrt().float() * weight
    h = c["rot"] // 2
    there = (positions >= 0)[:, None, None]
    cos, sin = s["table"][positions.clamp(min=0).long()][:, None].split(h, -1)
    turn = x[..., :2 * h]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if c["pairs"] else (turn[..., :h], turn[..., h:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turn = torch.stack([u, v], -1).flatten(-2) if c["pairs"] else torch.cat([u, v], -1)
    return torch.where(there, torch.cat([turn, x[..., 2 * h:]], -1), 0)


def _rope(s):
    t = getattr(torch, s["c"]["out"])
    return [_turned(s["Q"], s["q_norm"], s["positions"], s).to(t), _turned(s["K"], s["k_norm"], s["positions"], s).to(t)]


def _tree_positions(s):
    """Position of each node: the prefix and the node's depth, -1 past the request's nodes."""
    T = s["c"]["T"]
    up = torch.nn.functional.one_hot(s["parents"].clamp(min=0).long(), T).float()
    up[:, 0] = 0
    reach = torch.eye(T, device="cuda") + up
    reach = _closed(reach, max(1, (T - 1).bit_length()))
    depth = reach.sum(-1).int() - 1
    return torch.where(torch.arange(T, device="cuda")[None] < s["new"][:, None], s["prefix"][:, None] + depth, -1)


def _closed(reach, times):
    return reach if times == 0 else _closed((reach @ reach > 0).float(), times - 1)


def _quantise(x):
    """fp32 rows [..., d] -> codes uint8 [..., d/2] (halves not yet swapped) and bf16 parameters [..., 2]."""
    lo, hi = x.amin(-1), x.amax(-1)
    k = torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)
    s = (hi * k - lo * k).bfloat16().float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    z = (lo + 8 * s).bfloat16().float()
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    q = torch.where(s[..., None] > 0, (torch.round((x - z[..., None]) * inv[..., None]) + 8).clamp(0, 15), torch.full_like(x, 8)).to(torch.uint8)
    q = q.unflatten(-1, (-1, 4, 2))
    nib = torch.cat([q[..., 0], q[..., 1]], -1).unflatten(-1, (4, 2))
    return (nib[..., 0] | (nib[..., 1] << 4)).flatten(-2), torch.stack([s, z], -1).bfloat16()


def _values(codes, par):
    """fp32 values of code rows [..., d/2] (halves in order) with parameters [..., 2]."""
    w = codes.unflatten(-1, (-1, 4))
    nib = torch.stack([w & 15, w >> 4], -1).flatten(-2)
    q = torch.stack([nib[..., :4], nib[..., 4:]], -1).flatten(-3).float()
    return par[..., 1:2].float() + par[..., 0:1].float() * (q - 8)


def _row_halves(rows, at, d):
    """Code rows [n, Hkv, d/2] with their halves in the order of page row `at` (and back)."""
    if d != 128:
        return rows
    v = rows.unflatten(-1, (2, 32))
    return torch.where(((at >> 1) & 1).bool()[:, None, None, None], v.flip(-2), v).flatten(-2)


def _append(s):
    c = s["c"]
    P, d = c["page"], c["d"]
    at = (_tree_positions(s) if c["tree"] else s["positions"]).flatten()
    codes = s["pool"][..., :P * d].unflatten(-1, (2, P, d // 2))
    par = s["pool"][..., P * d:].unflatten(-1, (2, P, 4))
    there = s["slots"] >= 0
    slots = s["slots"].clamp(min=0).long()
    page, row = slots // P, slots % P
    back = []
    for which, x in enumerate((_turned(s["K"], s["k_norm"], at, s), s["V"].float())):
        q, p = _quantise(x[there])
        codes[page[there], :, which, row[there]] = _row_halves(q, row[there], d)
        par[page[there], :, which, row[there]] = p.view(torch.uint8)
        v = _values(_row_halves(codes[page, :, which, row], row, d), par[page, :, which, row].contiguous().view(torch.bfloat16))
        back.append(torch.where(there[:, None, None], v, torch.zeros_like(v)).bfloat16())
    q = _turned(s["Q"], s["q_norm"], at, s).bfloat16() if c["Hq"] else None
    return dict(Q=q, K=back[0], V=back[1])


def _prompt(s):
    c = s["c"]
    G, Hkv, L = c["Hq"] // c["Hkv"], c["Hkv"], s["longest"]
    i = torch.arange(L, device="cuda")
    n = (s["cu"][1:] - s["cu"][:-1])[:, None]
    there = i[None] < n                                                   # [B, L]
    at = torch.where(there, s["cu"][:-1, None] + i[None], 0).long()
    q = s["Q"].float()[at].unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, L, d]
    k, v = (x.float()[at].transpose(1, 2)[:, :, None] for x in (s["K"], s["V"]))
    x = (q * c["d"] ** -0.5) @ k.transpose(-1, -2)
    x.masked_fill_(i[None, :] > i[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (x @ v) / x.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(s["Q"].dtype)  # packed again


def _lora(s):
    a = s["ids"].clamp(min=0).long()
    t = (s["A"][a].float() @ s["X"].float()[:, :, None])[..., 0] * s["scale"][a][:, None]
    more = (s["B"][a].float() @ t[:, :, None])[..., 0]
    s["Y"] += torch.where(s["ids"][:, None] >= 0, more, 0)
    return s["Y"]


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope, "append": _append, "prompt": _prompt, "lora": _lora}[s["c"]["op"]](s)


def _run_own(s):
    from speculative_decoding_verification_w12_gb300 import w12
    c = s["c"]
    handle = s.get("handle")  # what a serving loop makes once and keeps: the binding's objects and workspace
    if c["op"] == "prompt":
        return w12.prompt_attention(s["Q"], s["K"], s["V"], s["cu"])
    if c["op"] == "lora":
        if handle is None:
            handle = s["handle"] = w12.LoRA(s["A"], s["B"], s["scale"])
        return handle.run(s["X"], s["Y"], s["ids"])
    if c["op"] == "rope":
        if handle is None:
            handle = s["handle"] = w12.Rope(s["table"], c["d"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, interleaved=c["pairs"])
        return list(handle.run(s["Q"], s["K"], s["positions"], dtype=getattr(torch, c["out"])))
    if handle is None:
        handle = s["handle"] = (w12.KV4Cache(s["pool"], c["page"], c["d"]),
                                w12.Rope(s["table"], c["d"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, interleaved=c["pairs"]))
    cache, rope = handle
    at = w12.tree_positions(s["prefix"], s["parents"], q_len=s["new"]) if c["tree"] else s["positions"]
    q = cache.append_rope(s["K"], s["V"], s["slots"], rope, at.flatten(), Q=s["Q"])
    k, v = cache.read(s["slots"])
    return dict(Q=q, K=k, V=v)


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_turned(x, weight, positions, c):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    out = x.clone()
    angle = positions.double()[:, None] * _inv_freq(c["rot"])
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["pairs"] else (slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"]))
    w = torch.complex(x[..., first], x[..., second]) * z
    out[..., first], out[..., second] = w.real, w.imag
    out[positions < 0] = 0
    return out


def _exact_row(x):
    """The values that rows [..., d] come back as from the cache."""
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).float().bfloat16().double()
    z = (lo + 8 * s).float().bfloat16().double()
    return z + s * (((x - z) / s).round() + 8).clamp(0, 15).sub(8)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return [_exact_turned(s["Q"], s["q_norm"], s["positions"], c), _exact_turned(s["K"], s["k_norm"], s["positions"], c)]
    if c["op"] == "append":
        at = torch.full((c["B"], c["T"]), -1, dtype=torch.int64, device="cuda")
        if c["tree"]:
            for b, parents in enumerate(s["parents"].tolist()):
                for t in range(int(s["new"][b])):
                    depth, i = 0, t
                    while parents[i] >= 0:
                        depth, i = depth + 1, parents[i]
                    at[b, t] = int(s["prefix"][b]) + depth
        else:
            at = s["positions"].long()
        at, out = at.flatten(), []
        for x in (_exact_turned(s["K"], s["k_norm"], at, c), s["V"].double()):
            v = _exact_row(x)
            v[s["slots"] < 0] = 0
            out.append(v)
        return dict(Q=_exact_turned(s["Q"], s["q_norm"], at, c) if c["Hq"] else None, K=out[0], V=out[1])
    if c["op"] == "prompt":
        G, cu = c["Hq"] // c["Hkv"], s["cu"].tolist()
        out = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
        for a, e in zip(cu, cu[1:]):
            hidden = torch.ones((e - a, e - a), dtype=torch.bool, device="cuda").triu(1)
            for h in range(c["Hq"] if e > a else 0):
                q, k, v = s["Q"][a:e, h].double(), s["K"][a:e, h // G].double(), s["V"][a:e, h // G].double()
                out[a:e, h] = torch.softmax((q @ k.T / math.sqrt(c["d"])).masked_fill(hidden, -math.inf), -1) @ v
        return out
    out = s["Y"].double()
    for m, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            out[m] += s["scale"][a].double() * (s["B"][a].double() @ (s["A"][a].double() @ s["X"][m].double()))
    return out
