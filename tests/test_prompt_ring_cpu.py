"""The prompt kernel's ring of key and value blocks, its barriers and its notes, played through on
the CPU with warps that run at any speed.

A barrier's wait names a parity alone: a warp that comes when the barrier is a phase further or a phase
behind passes at once, or never. So nothing but the order of arrivals may keep every wait on its own phase,
however late one warp is. Here each role of the kernel is a coroutine, each barrier counts its phases, and
whoever runs next is drawn with one of the roles held back. What the kernel waits for and how many
arrivals its barriers take is read from its source.
"""
import os
import random
import re

import pytest

from speculative_decoding_verification_w12_gb300 import build as B

SRC = open(os.path.join(B.CSRC, "w12_prompt.cu")).read()


class Stale(Exception):
    """A wait that passed on another phase than its own, or data that are not those meant."""


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passes(self, k):
        """Whether a wait for the parity of phase k returns."""
        if (self.phase & 1) == (k & 1):
            return False
        if self.phase != k + 1:
            raise Stale(f"wait for phase {k} passed while {self.phase} are complete")
        return True


def _count(name):
    return int(re.search(r"mbar_init\(&" + name + r"\[\w+\], (\d+)\)", SRC).group(1))


def rules():
    """From the source: what P V waits for, the places that are looked through, arrivals at a stage's release."""
    body = SRC[SRC.index("------ products"):SRC.index("------ softmax")]
    if re.search(r"ok = wait_all\(!is_s && j >= cut \? &clean\[s\] : &full\[s\]", body):
        waits = "cut"        # for the look at V where the diagonal cuts it, for the copy elsewhere
    elif re.search(r"ok = wait_all\(&full\[s\], (\w+)\) && \(is_s \|\| wait_all\(&clean\[s\], \1\)\)", body):
        waits = "all"        # for the copy, and of V for the look at it
    else:
        raise AssertionError("the products' wait is not one that this model knows")
    if re.search(r"for \(int place = base; place < base \+ 2 \* all; \+\+place\)", body):
        step = 1
    elif re.search(r"for \(int j = 0; ok && j < all; \+\+j, place \+= 2\)", body[body.index("not finite"):]):
        step = 2
    else:
        raise AssertionError("the walk of the warps that look through V is not one that this model knows")
    return waits, step


class Kernel:
    """One block of the kernel: items are (blocks of tile 0, blocks of tile 1, first cut block)."""
    kItems, kBadItems = 4, 8

    def __init__(self, items, stages, waits, step, rng):
        self.items, self.stages, self.waits, self.step, self.rng = items, stages, waits, step, rng
        b = lambda n, count: [Barrier(count) for _ in range(n)]  # noqa: E731
        self.full, self.empty, self.clean = b(stages, 1), b(stages, _count("empty")), b(stages, _count("clean"))
        self.q_full, self.q_empty, self.s_full, self.s_read, self.p_full, self.o_done, self.o_free = (b(2, 1) for _ in range(7))
        self.it_full, self.it_empty = b(self.kItems, 1), b(self.kItems, 9)   # readers of this model
        self.slots = [None] * self.kItems
        self.at = [None] * stages                 # the place whose block a stage holds
        self.looked = [set() for _ in range(stages)]
        self.notes = {}
        self.later = {}                           # copies and products under way, each series in order

    def get(self, k):
        yield self.it_full[k % 4], k // 4
        it = self.slots[k % 4]
        self.it_empty[k % 4].arrive()
        return it

    def hand_out(self):
        for k, it in enumerate(self.items + [None]):
            if k >= 4:
                yield self.it_empty[k % 4], k // 4 - 1
            self.slots[k % 4] = it if it is None else (k, *it)
            self.it_full[k % 4].arrive()

    def copy(self):
        issued, q = 0, [0, 0]

        def land(place):
            s = place % self.stages
            self.at[s], self.looked[s] = place, set()
            self.full[s].arrive()
        k = 0
        while (it := (yield from self.get(k))) is not None:
            n0, n1 = it[1:3]
            for place in range(2 * max(n0, n1)):
                if issued >= self.stages:
                    yield self.empty[issued % self.stages], issued // self.stages - 1
                self.later.setdefault("copies", []).append(lambda p=issued: land(p))
                issued += 1
                if place == 0:
                    for i in range(2 if n1 else 1):
                        if q[i]:
                            yield self.q_empty[i], q[i] - 1
                        self.later["copies"].append(self.q_full[i].arrive)
                        q[i] += 1
            k += 1

    def product(self, i, is_s):
        place, blocks, mine, k = 0 if is_s else 1, 0, 0, 0
        queue = self.later.setdefault((i, is_s), [])
        while (it := (yield from self.get(k))) is not None:
            item, n0, n1, cut = it
            n = (n0, n1)[i]
            if n and is_s:
                yield self.q_full[i], mine
            if n and not is_s and mine:
                yield self.o_free[i], mine - 1
            for j in range(max(n0, n1)):
                s, turn = place % self.stages, place // self.stages
                if self.waits == "all" or is_s or j < cut:
                    yield self.full[s], turn
                if not is_s and (self.waits == "all" or j >= cut):
                    yield self.clean[s], turn
                if j >= n:
                    self.empty[s].arrive()
                else:
                    if is_s:
                        if blocks:
                            yield self.s_read[i], blocks - 1
                    else:
                        yield self.p_full[i], blocks

                    def done(s=s, place=place, j=j, last=j == n - 1, cut=cut):
                        if self.at[s] != place or (not is_s and j >= cut and self.looked[s] != {0, 1}):
                            raise Stale(f"a product reads place {place}: the stage holds {self.at[s]}, looked through by {self.looked[s]}")
                        (self.s_full if is_s else self.o_done)[i].arrive()
                        self.empty[s].arrive()
                        if is_s and last:
                            self.q_empty[i].arrive()
                    queue.append(done)
                    blocks += 1
                place += 2
            mine += n > 0
            k += 1

    def look(self, w):
        place, k = 0 if self.step == 1 else 1, 0
        while (it := (yield from self.get(k))) is not None:
            item, n0, n1, cut = it
            for j in range(2 * max(n0, n1) // self.step):
                s = place % self.stages
                yield self.full[s], place // self.stages
                block, is_v = (j // 2, j & 1) if self.step == 1 else (j, 1)
                if is_v and block >= cut:
                    if self.at[s] != place:
                        raise Stale("another block is looked through")
                    self.looked[s].add(w)
                    self.notes[item % self.kBadItems, block - cut, w] = item
                self.clean[s].arrive()
                place += self.step
            k += 1

    def softmax(self, i):
        blocks, k = 0, 0
        while (it := (yield from self.get(k))) is not None:
            item, n0, n1, cut = it
            n = (n0, n1)[i]
            for j in range(n):
                yield self.s_full[i], blocks + j
                self.s_read[i].arrive()
                if j:
                    yield self.o_done[i], blocks + j - 1
                self.p_full[i].arrive()
            if n:
                yield self.o_done[i], blocks + n - 1
                for b in range(n - cut):
                    if any(self.notes.get((item % self.kBadItems, b, w)) != item for w in (0, 1)):
                        raise Stale("notes of another item")
                self.o_free[i].arrive()
            blocks += n
            k += 1

    def play(self, late):
        """Runs to the end; `late` runs where nothing else can, and now and then."""
        roles = {"items": self.hand_out(), "copy": self.copy(), "softmax 0": self.softmax(0), "softmax 1": self.softmax(1),
                 "look 0": self.look(0), "look 1": self.look(1)}
        for i in (0, 1):
            roles[f"S {i}"], roles[f"P V {i}"] = self.product(i, True), self.product(i, False)
        want = dict.fromkeys(roles)

        def ready(name):
            return want[name] is None or want[name][0].passes(want[name][1])
        while roles or any(self.later.values()):
            can = [name for name in roles if ready(name)] + [key for key, q in self.later.items() if q]
            if not can:
                raise Stale(f"nobody can go on: {sorted(roles)}")
            prompt = [name for name in can if name not in late] or can
            name = self.rng.choice(prompt if self.rng.random() < 0.998 else can)
            if name not in roles:
                self.later[name].pop(0)()
                continue
            try:
                want[name] = next(roles[name])
            except StopIteration:
                del roles[name], want[name]


LATE = [(), ("look 0",), ("look 1",), ("look 0", "look 1"), ("P V 0",), ("P V 1",), ("S 0",), ("softmax 0",), ("softmax 1",),
        ("copy",), ("copies",), ("items",), ((0, False),), ((1, True),)]


def _items(rng):
    """Long items with a few cut blocks, short ones, and items of one tile."""
    out = []
    for _ in range(14):
        n0 = rng.choice([1, 2, 3, 7, 14, 25])
        n1 = rng.choice([0, n0, n0 + 1, n0 + 2])
        out.append((n0, n1, max(0, max(n0, n1) - rng.randint(1, 5))))
    return out


@pytest.mark.parametrize("late", LATE, ids=str)
@pytest.mark.parametrize("stages", [8, 10])
def test_every_wait_is_for_its_own_phase(stages, late):
    waits, step = rules()
    for seed in range(12):
        rng = random.Random(seed)
        Kernel(_items(rng), stages, waits, step, rng).play(late)


def test_the_model_sees_waits_that_nothing_holds_back():
    """Looks at V that only the cut blocks wait for: a late warp is passed by."""
    found = 0
    for seed in range(12):
        rng = random.Random(seed)
        try:
            Kernel(_items(rng), 8, "cut", 1, rng).play(("look 0",))
        except Stale:
            found += 1
    assert found


def test_the_model_has_the_kernels_rings():
    assert [int(v) for v in re.search(r"kStages = kD == 128 \? (\d+) : (\d+)", SRC).groups()] == [8, 10]
    assert (_count("full"), _count("empty"), _count("clean")) == (1, 2, 2)
    assert int(re.search(r"kItems = (\d+)", SRC).group(1)) == Kernel.kItems
    assert int(re.search(r"kBadItems = (\d+)", SRC).group(1)) == Kernel.kBadItems
