"""Measured cases of the paged 4-bit key/value cache and of the token log probabilities.

Four groups of operators, as a serving program uses them around a verify step:

  pages      block tables and slot maps from request lengths: reserve the pages of a step's
             new tokens, then give back what the step did not keep;
  write      quantise new keys and values into their slots, move the accepted path behind
             the committed prefix (commit), read rows back;
  attention  queries of one token, a drafted block, a draft tree or a prompt chunk over the
             4-bit cache;
  logprobs   log probabilities of given tokens, entropy and top alternatives of logits rows.

``run`` computes the plain form (torch, fp32) unless ``own`` is set; then it makes the calls
of the framework's w12 binding. Both work on the same buffers.

The cache ("KV4"): a pool uint8 [n_pages, Hkv, page_bytes], page_bytes = P (d + 8) for pages
of P tokens and head dimension d. A page holds, per kv head: K codes [P, d/2], V codes
[P, d/2], K parameters [P, 2], V parameters [P, 2] (bf16 scale s and bf16 centre z). A row
stores x as z + s (q - 8), q in 0..15. Word w of a row's codes holds dims 8w..8w+7: nibble j
(j < 4) is dim 8w + 2j, nibble j + 4 is dim 8w + 2j + 1; with d = 128 the row's two 32-byte
halves are swapped in rows whose index in the page has bit 1 set. Slot = page P + row.
"""
import math
import random

import torch

own = False

VOCAB = 151936


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One verify step's pages: 16 requests with a 16-token block each, then the block is dropped.
        dict(name="pages-verify-16x16", op="pages", B=16, T=16, page=64, len_max=8192, prompt=False),
        # A batch of prompts admitted at once (ragged, up to 1024 tokens) and released.
        dict(name="pages-prompts-256x1024", op="pages", B=256, T=1024, page=16, len_max=1024, prompt=True),
        # A draft tree's keys and values from the fp32 output of the qkv product (a strided view of it),
        # quantised into the pages, the accepted path committed, the kept rows read back.
        dict(name="write-tree-4x64-f32", op="write", B=4, T=64, Hkv=8, d=128, page=64, dtype="float32", commit=True, strided=True),
        # A batch of small-head trees on short pages.
        dict(name="write-tree-16x48-d64", op="write", B=16, T=48, Hkv=2, d=64, page=16, dtype="bfloat16", commit=True, strided=False),
        # Prompts: 4 requests of up to 8192 tokens, cached and read back.
        dict(name="write-prompt-4x8192", op="write", B=4, T=8192, Hkv=8, d=128, page=64, dtype="bfloat16", commit=False, strided=False),
        # One request, one token, a short odd length: latency.
        dict(name="attn-decode-1x777", op="attention", B=1, T=1, Hq=40, Hkv=8, d=128, page=64, len_max=777, tree=False, ragged=False),
        # Single tokens of a ragged batch (some slots idle).
        dict(name="attn-decode-64x8192", op="attention", B=64, T=1, Hq=40, Hkv=8, d=128, page=16, len_max=8192, tree=False, ragged=True),
        # Drafted 16-token blocks of 16 requests.
        dict(name="attn-block-16x16x8192", op="attention", B=16, T=16, Hq=40, Hkv=8, d=128, page=64, len_max=8192, tree=False, ragged=False),
        # 64-node draft trees of 4 requests over long caches.
        dict(name="attn-tree-4x64x32768", op="attention", B=4, T=64, Hq=40, Hkv=8, d=128, page=128, len_max=32768, tree=True, ragged=False),
        # Prompt chunks behind a cached prefix, ragged, 64-wide heads.
        dict(name="attn-prompt-2x2048-d64", op="attention", B=2, T=2048, Hq=32, Hkv=8, d=64, page=32, len_max=2000, tree=False, ragged=True),
        # The verified rows of one block; half the vocabulary masked.
        dict(name="logprobs-16-f32", op="logprobs", M=16, V=VOCAB, n=1, k=20, dtype="float32", masked=True, scale=1.0),
        # Rows of a large batch in bf16 (many ties), with a temperature.
        dict(name="logprobs-256-bf16", op="logprobs", M=256, V=VOCAB, n=4, k=8, dtype="bfloat16", masked=False, scale=1.25),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "write", "attention", "attention", "logprobs"])
    if op == "pages":
        if rng.random() < 0.5:
            return dict(op=op, B=_logint(rng, 1, 256), T=_logint(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), len_max=_logint(rng, 16, 8192), prompt=False)
        T = _logint(rng, 16, 1024)
        return dict(op=op, B=_logint(rng, 1, 256), T=T, page=rng.choice([16, 32, 64, 128]), len_max=T, prompt=True)
    if op == "write":
        heads = dict(Hkv=rng.choice([1, 2, 4, 5, 8]), d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["float32", "bfloat16", "float16"]))
        if rng.random() < 0.6:
            return dict(op=op, B=_logint(rng, 1, 16), T=_logint(rng, 1, 64), commit=True, strided=rng.random() < 0.5, **heads)
        return dict(op=op, B=rng.randint(1, 4), T=_logint(rng, 65, 8191), commit=False, strided=rng.random() < 0.5, **heads)
    if op == "attention":
        kind = rng.choice(["decode", "block", "tree", "prompt"])
        T = {"decode": 1, "block": rng.randint(2, 16), "tree": rng.randint(17, 64), "prompt": _logint(rng, 100, 2048)}[kind]
        Hq, Hkv = rng.choice([(40, 8), (32, 8), (16, 2), (8, 8), (10, 2), (12, 4), (16, 1)])
        c = dict(op=op, B=_logint(rng, 1, {"decode": 64, "block": 16, "tree": 4, "prompt": 2}[kind]), T=T, Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), len_max=_logint(rng, 1, 2048 if kind == "prompt" else 32768), tree=kind == "tree" or (kind == "block" and rng.random() < 0.5),
                 ragged=rng.random() < 0.6)
        most = [work(x) for x in listed() if x["op"] == "attention"]
        while work(c)["bytes"] > max(w["bytes"] for w in most) or work(c)["flops"] > max(w["flops"] for w in most):
            c["len_max"] = max(1, c["len_max"] * 2 // 3)
        return c
    return dict(op=op, M=_logint(rng, 1, 256), V=rng.choice([VOCAB, 32000, 4096, _logint(rng, 2, 150001)]), n=rng.randint(1, 4), k=rng.choice([0, 1, 5, 8, 20, 32]),
                dtype=rng.choice(["float32", "bfloat16", "float16"]), masked=rng.random() < 0.4, scale=rng.choice([1.0, 0.7, 1.25]))


def _lengths(c):
    """(tokens already cached, new tokens) of each request: plain lists, from the case alone."""
    cached, new = [], []
    for b in range(c["B"]):
        f = ((b + 1) * 0.6180339887498949) % 1.0
        if c["op"] == "pages":
            if c["prompt"]:
                cached.append(0)
                new.append(1 + int(f * c["T"] * 0.999))
            else:
                cached.append(1 + int(f * (c["len_max"] - 1)))
                new.append(c["T"])
        elif c["op"] == "write":
            cached.append(int(f * 700) if c["commit"] else 0)
            new.append(c["T"] if c["commit"] else c["T"] - int(f * c["T"] / 4))
        elif c["ragged"]:
            cached.append(c["len_max"] // 4 + int(f * (c["len_max"] - c["len_max"] // 4)))
            new.append(0 if b % 16 == 7 else c["T"] - int(f * (c["T"] // 2)))
        else:
            cached.append(c["len_max"])
            new.append(c["T"])
    return cached, new


def work(c):
    cached, new = _lengths(c) if c["op"] != "logprobs" else ([], [])
    if c["op"] == "pages":
        # Slots written once, lengths read; the pages that change hands are read and written once each way.
        moved = sum(-(-(a + n) // c["page"]) - -(-a // c["page"]) for a, n in zip(cached, new))
        return dict(bytes=4 * c["B"] * c["T"] + 24 * c["B"] + 16 * moved, flops=4 * c["B"] * c["T"])
    if c["op"] == "write":
        rows, e = sum(new) * c["Hkv"], 4 if c["dtype"] == "float32" else 2
        moves = 2 * sum(min(_depth(c), n) for n in new) * c["Hkv"] * (c["d"] + 8) if c["commit"] else 0
        return dict(bytes=rows * (2 * c["d"] * e + 2 * (c["d"] + 8) + 4 * c["d"]) + moves, flops=rows * 2 * c["d"] * 8)
    if c["op"] == "attention":
        G, d = c["Hq"] // c["Hkv"], c["d"]
        keys = sum(a + n for a, n in zip(cached, new) if n)
        seen = sum(n * a + n * (n + 1) // 2 for a, n in zip(cached, new))
        return dict(bytes=keys * c["Hkv"] * (d + 8) + 4 * sum(new) * c["Hq"] * d + 2 * (c["B"] * c["T"] - sum(new)) * c["Hq"] * d,
                    flops=4 * seen * c["Hkv"] * G * d)
    e = 4 if c["dtype"] == "float32" else 2
    return dict(bytes=c["M"] * (c["V"] * e + 8 * c["n"] + 8 * c["k"] + 8), flops=4 * c["M"] * c["V"])


def _depth(c):
    """Accepted nodes of a committed path (the root among them)."""
    return max(1, min(7, c["T"]))


# ------------------------------------------------------------------ inputs
def _tree(r, T, deep):
    """Parents of a T-node draft tree whose first `deep` levels exist (node 0 is the root)."""
    parents = [-1]
    for i in range(1, T):
        parents.append(r.randrange(i) if r.random() < 0.7 else i - 1)
    path = list(range(0, T, max(1, T // deep)))[:deep]
    for a, b in zip(path, path[1:]):
        parents[b] = a
    return parents, path


def _halves(codes, d):
    """Swap the 32-byte halves of rows with bit 1 of their page row set: codes [..., P, d/2], d = 128."""
    if d != 128:
        return codes
    v = codes.unflatten(-1, (2, 32))
    odd = ((torch.arange(codes.shape[-2], device=codes.device) >> 1) & 1).bool()
    return torch.where(odd[:, None, None], v.flip(-2), v).flatten(-2)


def _quantise(x):
    """fp32 rows [..., d] -> codes uint8 [..., d/2] (rows not yet swapped) and bf16 parameters [..., 2]."""
    lo, hi = x.amin(-1), x.amax(-1)
    r = torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)
    s = (hi * r - lo * r).bfloat16().float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    z = (lo + 8 * s).bfloat16().float()
    bad = ~torch.isfinite(hi * 0 + lo * 0)
    s, z = torch.where(bad, float("nan"), s), torch.where(bad, float("nan"), z)
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    q = torch.where(s[..., None] > 0, (torch.round((x - z[..., None]) * inv[..., None]) + 8).clamp(0, 15), torch.full_like(x, 8)).to(torch.uint8)
    q = q.unflatten(-1, (-1, 4, 2))                                   # word, j, (dim 2j, dim 2j + 1)
    nib = torch.cat([q[..., 0], q[..., 1]], -1).unflatten(-1, (4, 2))  # nibbles 0..7 of each word
    return (nib[..., 0] | (nib[..., 1] << 4)).flatten(-2), torch.stack([s, z], -1).bfloat16()


def _values(codes, par):
    """fp32 values of code rows (already unswapped) [..., d/2] with parameters [..., 2]."""
    w = codes.unflatten(-1, (-1, 4))
    nib = torch.stack([w & 15, w >> 4], -1).flatten(-2)                # nibbles 0..7
    q = torch.stack([nib[..., :4], nib[..., 4:]], -1).flatten(-3).float()
    return par[..., 1:2].float() + par[..., 0:1].float() * (q - 8)


def _parts(pages, d):
    """K codes, V codes (unswapped), K and V parameters of pages uint8 [..., Hkv, P (d + 8)]."""
    P = pages.shape[-1] // (d + 8)
    codes = pages[..., :P * d].unflatten(-1, (2, P, d // 2))
    par = pages[..., P * d:].contiguous().view(torch.bfloat16).unflatten(-1, (2, P, 2))
    return _halves(codes[..., 0, :, :], d), _halves(codes[..., 1, :, :], d), par[..., 0, :, :], par[..., 1, :, :]


def _fill(pool, table, lens, d, g):
    """Pool pages of every request's first `lens` tokens from N(0, 1) keys and values; all other rows hold 0xFF."""
    n_pages, Hkv, pb = pool.shape
    P = pb // (d + 8)
    pool.fill_(255)
    step = max(1, (1 << 27) // (Hkv * P * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        out = []
        for _ in range(2):
            codes, par = _quantise(torch.randn((n, Hkv, P, d), generator=g, device=pool.device))
            out.append((_halves(codes, d).flatten(-2), par.view(torch.uint8).flatten(-2)))
        pool[i:i + n] = torch.cat([out[0][0], out[1][0], out[0][1], out[1][1]], -1)
    # Rows past each request's length, in its last page: parameters no one may use.
    for b, L in enumerate(lens):
        if L % P:
            par = pool[int(table[b][L // P]), :, P * d:].unflatten(-1, (2, P, 4))
            par[:, :, L % P:] = 255


def _tables(r, need, B, spare=3):
    """Pages of each request in shuffled order: table as lists, page count, free pages."""
    total = sum(need) + spare
    ids = list(range(total))
    r.shuffle(ids)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n])
        at += n
    return table, total, ids[at:]


def _table_tensor(table, width):
    return torch.tensor([t + [-1] * (width - len(t)) for t in table], dtype=torch.int32, device="cuda")


def prepare(c, seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] == "logprobs":
        x = torch.randn((c["M"], c["V"] + 8), generator=g, device="cuda") * 2.5
        if c["masked"]:
            x[torch.rand(x.shape, generator=g, device="cuda") < 0.5] = -math.inf
        x = x.to(getattr(torch, c["dtype"]))[:, :c["V"]]  # rows padded to a longer pitch, as a logits buffer is
        tokens = torch.randint(0, c["V"], (c["M"], c["n"]), generator=g, device="cuda", dtype=torch.int32)
        return dict(c=c, logits=x, tokens=tokens)
    cached, new = _lengths(c)
    P, B, T = c["page"], c["B"], c["T"]
    pages_of = lambda n: -(-n // P)  # noqa: E731
    if c["op"] == "pages":
        used = [pages_of(n) for n in cached]
        width = max(pages_of(a + n) for a, n in zip(cached, new)) + 1
        grown = sum(pages_of(a + n) for a, n in zip(cached, new)) - sum(used)
        table, total, free = _tables(r, used, B, grown + 5)
        return dict(c=c, start=i32(cached), new=i32(new), table=_table_tensor(table, width), used=i32(used),
                    free=i32(free + [0] * (total - len(free))), n_free=i32([len(free)]))
    Hkv, d = c["Hkv"], c["d"]
    lens = [a + n for a, n in zip(cached, new)]
    table, total, _ = _tables(r, [pages_of(n) for n in lens], B)
    width = max(1, max(len(t) for t in table))
    pool = torch.empty((total, Hkv, P * (d + 8)), dtype=torch.uint8, device="cuda")
    s = dict(c=c, pool=pool, table=_table_tensor(table, width), prefix=i32(cached), new=i32(new))
    if c["op"] == "write":
        pool.fill_(0)
        slots = [[t[(a + i) // P] * P + (a + i) % P for i in range(n)] + [-1] * (T - n) for t, a, n in zip(table, cached, new)]
        wide = torch.randn((B * T, (c["Hkv"] * 4 if c["strided"] else c["Hkv"] * 2) * d), generator=g, device="cuda").to(getattr(torch, c["dtype"]))
        at = 2 * Hkv * d if c["strided"] else 0  # behind the queries of the same product
        s["K"] = wide[:, at:at + Hkv * d].unflatten(-1, (Hkv, d))
        s["V"] = wide[:, at + Hkv * d:at + 2 * Hkv * d].unflatten(-1, (Hkv, d))
        s["slots"] = i32(slots).flatten()
        if c["commit"]:
            paths = [_tree(r, T, _depth(c))[1] for _ in range(B)]
            shift = [[p[0]] + [x + r.randrange(0, max(1, T // _depth(c) - 1)) for x in p[1:]] for p in paths]
            paths = [[min(x, T - 1 - (len(p) - 1 - k)) for k, x in enumerate(p)] for p in shift]
            n = [r.randint(1, len(p)) for p in paths]
            s["path"] = i32([p + [-1] * (T - len(p)) for p in paths])
            s["path_len"] = i32(n)
        return s
    _fill(pool, table, lens, d, g)
    s["Q"] = torch.randn((B, T, c["Hq"], d), generator=g, device="cuda").bfloat16()
    s["parents"] = i32([_tree(r, T, min(12, T))[0] for _ in range(B)]) if c["tree"] else None
    s["max_len"] = max(lens)
    return s


# ------------------------------------------------------------------ plain forms
def _pages_update(s, start, new, T):
    """Table, counts and free stack brought to ceil((start + new) / P) pages a request; slots of the new tokens."""
    P, table, used, free, n_free = s["c"]["page"], s["table"], s["used"], s["free"], s["n_free"]
    want = (start + new + P - 1) // P
    grow = (want - used).clamp(min=0)
    upto = torch.cumsum(grow, 0)
    ok = (upto <= n_free) | (grow == 0)
    before = upto - grow
    grow = torch.where(ok, grow, torch.zeros_like(grow))
    shrink = (used - want).clamp(min=0)
    ahead = torch.cumsum(shrink, 0) - shrink
    G, R = grow.sum(), shrink.sum()
    j = torch.arange(table.shape[1], device="cuda")[None]
    taken = (j >= used[:, None]) & (j < want[:, None]) & ok[:, None]
    k = (n_free - 1 - (before[:, None] + j - used[:, None])).clamp(0, free.numel() - 1)
    got = torch.where(taken, free[k.long()], table)
    back = (j >= want[:, None]) & (j < used[:, None])
    at = torch.where(back, n_free - G + R - 1 - (ahead[:, None] + j - want[:, None]), torch.full_like(got, free.numel()).long())
    more = torch.cat([free, free.new_zeros(1)])
    more.scatter_(0, at.flatten().long(), table.flatten())
    free.copy_(more[:-1])
    table.copy_(torch.where(back, torch.full_like(got, -1), got))
    n_free.copy_(n_free + R - G)
    used.copy_(torch.where(ok, want, used))
    i = torch.arange(T, device="cuda")[None]
    pos = start[:, None] + i
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1).long())
    return torch.where((i < new[:, None]) & ok[:, None], page * P + (pos % P).int(), torch.full_like(page, -1))


def _views(s):
    """The pool's K codes, V codes, K and V parameters as [n_pages, Hkv, P, bytes] views."""
    d, P = s["c"]["d"], s["c"]["page"]
    codes = s["pool"][..., :P * d].unflatten(-1, (2, P, d // 2))
    par = s["pool"][..., P * d:].unflatten(-1, (2, P, 4))
    return codes[:, :, 0], codes[:, :, 1], par[:, :, 0], par[:, :, 1]


def _row_halves(rows, row_in_page, d):
    """_halves() of code rows [n, Hkv, d/2] that sit at the given page rows."""
    if d != 128:
        return rows
    v = rows.unflatten(-1, (2, 32))
    return torch.where(((row_in_page >> 1) & 1).bool()[:, None, None, None], v.flip(-2), v).flatten(-2)


def _append(s):
    P, d = s["c"]["page"], s["c"]["d"]
    valid = s["slots"] >= 0
    slots = s["slots"][valid].long()
    page, row = slots // P, slots % P
    kc, vc, kp, vp = _views(s)
    for x, codes, par in ((s["K"], kc, kp), (s["V"], vc, vp)):
        q, p = _quantise(x[valid].float())
        codes[page, :, row] = _row_halves(q, row, d)
        par[page, :, row] = p.view(torch.uint8)


def _commit(s):
    P, d, T = s["c"]["page"], s["c"]["d"], s["c"]["T"]
    k = torch.arange(T, device="cuda")[None]
    live = k < s["path_len"][:, None]
    slot = lambda pos: (s["table"].gather(1, (pos // P).long()).long() * P + pos % P)[live]  # noqa: E731
    src, dst = slot(torch.where(live, s["prefix"][:, None] + s["path"], 0)), slot(torch.where(live, s["prefix"][:, None] + k, 0))
    kc, vc, kp, vp = _views(s)
    for codes in (kc, vc):
        codes[dst // P, :, dst % P] = _row_halves(_row_halves(codes[src // P, :, src % P], src % P, d), dst % P, d)
    for par in (kp, vp):
        par[dst // P, :, dst % P] = par[src // P, :, src % P]


def _read(s):
    P, d = s["c"]["page"], s["c"]["d"]
    slots = s["slots"].clamp(min=0).long()
    page, row = slots // P, slots % P
    kc, vc, kp, vp = _views(s)
    out = []
    for codes, par in ((kc, kp), (vc, vp)):
        x = _values(_row_halves(codes[page, :, row], row, d), par[page, :, row].contiguous().view(torch.bfloat16))
        out.append(torch.where((s["slots"] >= 0)[:, None, None], x, torch.zeros_like(x)).bfloat16())
    return out


def _seen(s, keys):
    """[B, T, keys]: whether query t sees the key; by the causal order, or by its path in the draft tree."""
    c = s["c"]
    B, T = c["B"], c["T"]
    t, j = torch.arange(T, device="cuda"), torch.arange(keys, device="cuda")
    rel = j[None, :] - s["prefix"][:, None].long()                       # draft index of a key
    live = (t[None] < s["new"][:, None])[:, :, None]
    if s["parents"] is None:
        return live & (rel[:, None, :] <= t[None, :, None])
    up = torch.nn.functional.one_hot(s["parents"].clamp(min=0).long(), T).float()
    up[:, 0] = 0
    anc = torch.eye(T, device="cuda").expand(B, T, T) + up
    for _ in range(max(1, (T - 1).bit_length())):                         # reachability by squaring
        anc = (anc @ anc > 0).float()
    tree = torch.cat([anc.bool(), torch.zeros((B, T, 1), dtype=torch.bool, device="cuda")], 2)
    own_path = tree.gather(2, torch.where((rel >= 0) & (rel < T), rel, T)[:, None, :].expand(B, T, keys))
    return live & ((rel < 0)[:, None, :] | own_path)


def _attention(s):
    c = s["c"]
    d, Hkv, B, T = c["d"], c["Hkv"], c["B"], c["T"]
    G = c["Hq"] // Hkv
    pages = s["pool"][s["table"].clamp(min=0).long()]                     # [B, width, Hkv, page bytes]
    kc, vc, kp, vp = _parts(pages, d)
    flat = lambda x: x.transpose(1, 2).flatten(2, 3)                      # noqa: E731  [B, Hkv, keys, d]
    K, V = flat(_values(kc, kp)), flat(_values(vc, vp))
    keys = K.shape[2]
    there = (torch.arange(keys, device="cuda")[None] < (s["prefix"] + s["new"])[:, None])[:, None, :, None]
    K, V = torch.where(there, K, 0), torch.where(there, V, 0)
    Q = s["Q"].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = (Q @ K.transpose(-1, -2)) * d ** -0.5
    x = x.unflatten(2, (G, T)).masked_fill(~_seen(s, keys)[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ V).unflatten(2, (G, T)) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).bfloat16()


def _logprobs(s):
    c = s["c"]
    x = s["logits"].float() * c["scale"]
    top = x.amax(-1, keepdim=True)
    t = x - torch.where(top == -math.inf, 0, top)
    e = torch.exp(t)
    total = e.sum(-1, keepdim=True)
    nothing = top[:, 0] == -math.inf  # every token of the row is masked
    entropy = torch.where(nothing, 0, total.log()[:, 0] - (e * t.clamp(min=-1e30)).sum(-1) / total[:, 0])
    lse = (top + total.log())[:, 0]
    lp = torch.where(nothing[:, None], -math.inf, x.gather(1, s["tokens"].long()) - lse[:, None])
    values, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    k = min(c["k"], c["V"])
    values, ids = values[:, :k], ids[:, :k].int()
    ids = torch.where(values == -math.inf, -1, ids)
    pad = c["k"] - k  # more alternatives asked for than there are tokens
    values = torch.where(nothing[:, None], -math.inf, values - lse[:, None])
    values = torch.nn.functional.pad(values, (0, pad), value=-math.inf)
    return dict(logprob=lp, entropy=entropy, lse=lse, top_logprob=values, top_id=torch.nn.functional.pad(ids, (0, pad), value=-1))


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        return _run_own(s)
    if c["op"] == "pages":
        slots = _pages_update(s, s["start"], s["new"], c["T"])
        _pages_update(s, s["start"], torch.zeros_like(s["new"]), 0)
        return dict(slots=slots, table=s["table"], used=s["used"], free=s["free"], n_free=s["n_free"])
    if c["op"] == "write":
        _append(s)
        if c["commit"]:
            _commit(s)
        return _read(s)
    if c["op"] == "attention":
        return _attention(s)
    return _logprobs(s)


def _run_own(s):
    from speculative_decoding_verification_w12_gb300 import w12
    c = s["c"]
    handle = s.get("handle")  # what a serving loop makes once and keeps: the binding's plan and workspace
    if c["op"] == "pages":
        if handle is None:
            handle = s["handle"] = w12.PageTable(s["table"], s["used"], s["free"], s["n_free"], c["page"])
        slots = handle.reserve(s["start"], s["new"], c["T"])
        handle.trim(s["start"])
        return dict(slots=slots, table=s["table"], used=s["used"], free=s["free"], n_free=s["n_free"])
    if c["op"] == "write":
        if handle is None:
            handle = s["handle"] = w12.KV4Cache(s["pool"], c["page"], c["d"])
        handle.append(s["K"], s["V"], s["slots"])
        if c["commit"]:
            w12.kv4_commit([handle], s["table"], s["prefix"], s["path"], s["path_len"])
        return list(handle.read(s["slots"]))
    if c["op"] == "attention":
        if handle is None:
            cache = w12.KV4Cache(s["pool"], c["page"], c["d"])
            handle = s["handle"] = (cache, w12.KV4Attention(c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["page"], s["max_len"]))
        return handle[1].run(s["Q"], handle[0], s["table"], s["prefix"], parents=s["parents"], q_len=s["new"])
    if handle is None:
        handle = s["handle"] = w12.TokenLogprobs(c["M"], c["V"], c["k"])
    lp, entropy, lse, top_lp, top_id = handle.run(s["logits"], s["tokens"], scale=c["scale"])
    return dict(logprob=lp, entropy=entropy, lse=lse, top_logprob=top_lp, top_id=top_id)


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_row(x):
    """The values that a row of a tensor [..., d] comes back as from the cache."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).float().bfloat16().double()
    z = (lo + 8 * s).float().bfloat16().double()
    return z + s * (((x - z) / s).round() + 8).clamp(0, 15).sub(8) if bool((s > 0).all()) else None


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "pages":
        return None  # whole numbers: they have to be equal
    if c["op"] == "write":
        # Rows as appended, then the committed ones in their new places.
        out = []
        for x in (s["K"], s["V"]):
            v = _exact_row(x)
            if v is None:
                return None
            v = v.unflatten(0, (c["B"], c["T"])).clone()
            for b in range(c["B"]):
                if c["commit"]:
                    n = int(s["path_len"][b])
                    v[b, :n] = v[b, s["path"][b, :n].long()].clone()
                v[b, int(s["new"][b]):] = 0
            out.append(v.flatten(0, 1))
        return out
    if c["op"] == "attention":
        G, d, P = c["Hq"] // c["Hkv"], c["d"], c["page"]
        out = torch.zeros((c["B"], c["T"], c["Hq"], d), dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            n, a = int(s["new"][b]), int(s["prefix"][b])
            if n == 0:
                continue
            L = a + n
            pos = torch.arange(L, device="cuda")
            at = s["table"][b][pos // P].long()
            parents = None if s["parents"] is None else s["parents"][b].tolist()
            see = torch.zeros((n, L), dtype=torch.bool, device="cuda")
            for t in range(n if parents else 0):
                see[t, :a] = True
                i = t
                while i >= 0:
                    see[t, a + i] = True
                    i = parents[i]
            if not parents:
                see = pos[None, :] <= a + torch.arange(n, device="cuda")[:, None]
            for h in range(c["Hkv"]):
                kv = []
                for which in (0, 1):
                    base = which * P * d // 2 + (pos % P) * (d // 2)
                    dim = torch.arange(d, device="cuda")
                    nib = (dim % 8) // 2 + 4 * (dim % 2)
                    byte = (dim // 8) * 4 + nib // 2
                    where = byte[None] ^ ((((pos % P) >> 1) & 1) * 32)[:, None] if d == 128 else byte[None].expand(L, d)
                    raw = s["pool"][at[:, None], h, base[:, None] + where].int()
                    q = (raw >> (4 * (nib % 2))[None]) & 15
                    word = P * d + which * 4 * P + (pos % P) * 4
                    par = [(s["pool"][at, h, word + o].int() + 256 * s["pool"][at, h, word + o + 1].int()) for o in (0, 2)]
                    sc, ce = [((p << 16).view(torch.float32)).double() for p in par]
                    kv.append(ce[:, None] + sc[:, None] * (q.double() - 8))
                q = s["Q"][b, :n, h * G:(h + 1) * G].double()
                for i in range(G):
                    x = torch.where(see, q[:, i] @ kv[0].T / math.sqrt(d), -math.inf)
                    out[b, :n, h * G + i] = torch.softmax(x, -1) @ kv[1]
        return out
    x = s["logits"].double() * torch.tensor(c["scale"], dtype=torch.float32).double().item()
    lse = torch.logsumexp(x, -1)
    lp = torch.where(torch.isneginf(lse)[:, None], -math.inf, x - lse[:, None])
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp.clamp(min=-1e300), 0).sum(-1)
    k = min(c["k"], c["V"])
    top = torch.nn.functional.pad(lp.sort(-1, descending=True).values[:, :k], (0, c["k"] - k), value=-math.inf)
    return dict(logprob=lp.gather(1, s["tokens"].long()), entropy=entropy, lse=lse, top_logprob=top, top_id=None)
