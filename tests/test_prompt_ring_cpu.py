"""A model of the bf16 prompt kernel's barriers (``csrc/prompt_tc.cu``), run with copies landing in random order.

The warps of ``k_prompt_tc`` are written out here as Python generators that take the same steps in the same order: the
TMA warp, the gate warp, the MMA warp and the eight softmax warps.  A scheduler picks at random who goes on, which copy
lands next and when the tensor cores take their next instruction (they work in the order of issue).  Every read checks
what it finds: the ring slots, Q, the scores, P and the output hold exactly the tile that the reader means.  A wait that
never ends is a deadlock and fails too.

``kept_first=False`` is a form that is wrong on purpose: first key tiles land on their slots' own barriers, and the gate
warp passes them unwaited.  The model has to catch that one, or it catches nothing.
"""
import random

import pytest

FIRST = 8  # barriers for first key tiles (kFirst)


class Wrong(Exception):
    pass


class Bar:
    """An mbarrier: `phase` phases are complete; the next one needs `count` arrivals and all announced copies."""

    def __init__(self, count=1):
        self.count, self.left, self.copies, self.phase = count, count, 0, 0

    def _settle(self):
        if self.left < 0:
            raise Wrong("more arrivals than a phase has")
        if self.left == 0 and self.copies == 0:
            self.left, self.phase = self.count, self.phase + 1

    def arrive(self, copies=0):
        self.copies += copies
        self.left -= 1
        self._settle()

    def landed(self):
        self.copies -= 1
        self._settle()

    def done(self, parity):  # try_wait.parity
        return (self.phase & 1) != parity


class Cta:
    """`items`: key tiles of group 0 and of group 1 per item (pair: two query tiles, with keys of their own)."""

    def __init__(self, items, stages, pair, rng, kept_first=True):
        self.items, self.n, self.pair, self.rng, self.kept_first = items, stages, pair, rng, kept_first
        self.full, self.empty = [Bar() for _ in range(stages)], [Bar() for _ in range(stages)]
        self.first = [Bar() for _ in range(FIRST)]
        self.q_full, self.q_empty, self.s_full, self.o_done = ([Bar(), Bar()] for _ in range(4))
        self.p_full, self.drain = [Bar(5), Bar(5)], Bar()
        self.ring, self.q = [None] * stages, [None, None]
        self.s, self.p = [None, None], [[None] * 4, [None] * 4]
        self.o = [[], []]
        self.flying, self.pipe = [], []
        self.written = {}

    # ---- asynchronous copies and the tensor cores' queue
    def copy(self, bar, where, at, what):
        bar.arrive(copies=1)
        where[at] = "in flight"
        self.flying.append((bar, where, at, what))

    def land(self):
        bar, where, at, what = self.flying.pop(self.rng.randrange(len(self.flying)))
        where[at] = what
        bar.landed()

    def expect(self, found, wanted, what):
        if found != wanted:
            raise Wrong(f"{what}: {found} where {wanted} is meant")

    def mma_s(self, g, slot, j, i):
        def run():
            self.expect(self.ring[slot], ("K", j, g if self.pair else 0, i), "K")
            self.expect(self.q[g], j, "Q")
            self.s[g] = (j, i)
            self.p[g] = [None] * 4
        self.pipe.append(run)

    def mma_o(self, g, slot, j, i):
        def run():
            self.expect(self.ring[slot], ("V", j, g if self.pair else 0, i), "V")
            self.expect(self.p[g], [(j, i)] * 4, "P")
            self.o[g] = (self.o[g] if i > 0 else []) + [(j, i)]
        self.pipe.append(run)

    def commit(self, bar):
        self.pipe.append(bar.arrive)

    # ---- the warps; each yields (barrier, parity) to wait, None to let others go on
    def producer(self):
        slot = turn = firsts = 0
        qturn, uses = [0, 0], [0] * self.n

        def load(what, first):
            nonlocal slot, turn, firsts
            if turn > 0:
                yield self.empty[slot], (turn - 1) & 1
            own = first and self.kept_first
            self.copy(self.first[firsts % FIRST] if own else self.full[slot], self.ring, slot, what)
            if own:
                firsts += 1
            else:
                uses[slot] += 1
            slot, turn = (0, turn + 1) if slot + 1 == self.n else (slot + 1, turn)
            yield None

        def load_q(g, j):
            if qturn[g] > 0:
                yield self.q_empty[g], (qturn[g] - 1) & 1
            self.copy(self.q_full[g], self.q, g, j)
            qturn[g] += 1
            yield None

        for j, nt in enumerate(self.items):
            if self.pair:
                for g in range(2):
                    if nt[g]:
                        yield from load_q(g, j)
                        yield from load(("K", j, g, 0), True)
                for i in range(max(nt)):
                    for g in range(2):
                        if i < nt[g]:
                            yield from load(("V", j, g, i), False)
                            if i + 1 < nt[g]:
                                yield from load(("K", j, g, i + 1), False)
            else:
                if nt[0]:
                    yield from load_q(0, j)
                if max(nt):
                    yield from load(("K", j, 0, 0), True)
                if nt[1]:
                    yield from load_q(1, j)
                for i in range(max(nt)):
                    yield from load(("V", j, 0, i), False)
                    if i + 1 < max(nt):
                        yield from load(("K", j, 0, i + 1), False)
        for g in range(2):
            if qturn[g]:
                yield self.q_full[g], (qturn[g] - 1) & 1
        for s in range(self.n):
            if uses[s]:
                yield self.full[s], (uses[s] - 1) & 1
        for i in range(FIRST):
            n = (firsts + FIRST - 1 - i) // FIRST
            if n:
                yield self.first[i], (n - 1) & 1

    def gate(self):
        slot, phase, pturn = 0, [0] * self.n, [0, 0]

        def advance():
            nonlocal slot
            if not self.kept_first:
                phase[slot] ^= 1  # the slot's phase goes by, landed or not
            slot = (slot + 1) % self.n

        def wait_full(what):
            nonlocal slot
            yield self.full[slot], phase[slot]
            self.expect(self.ring[slot], what, "gate")  # (it writes zeros behind a sequence's end here)
            phase[slot] ^= 1
            slot = (slot + 1) % self.n

        def arrive(g):
            if pturn[g] > 0:
                yield self.p_full[g], (pturn[g] - 1) & 1
            self.p_full[g].arrive()
            pturn[g] += 1
            yield None

        for j, nt in enumerate(self.items):
            if self.pair:
                for g in range(2):
                    if nt[g]:
                        advance()
                for i in range(max(nt)):
                    for g in range(2):
                        if i < nt[g]:
                            yield from wait_full(("V", j, g, i))
                            if i + 1 < nt[g]:
                                yield from wait_full(("K", j, g, i + 1))
                            yield from arrive(g)
            else:
                if max(nt):
                    advance()
                for i in range(max(nt)):
                    yield from wait_full(("V", j, 0, i))
                    if i + 1 < max(nt):
                        yield from wait_full(("K", j, 0, i + 1))
                    for g in range(2):
                        if i < nt[g]:
                            yield from arrive(g)

    def mma(self):
        slot, firsts, qturn, pturn, phase = 0, 0, [0, 0], [0, 0], [0] * self.n

        def advance():
            nonlocal slot
            s, slot = slot, (slot + 1) % self.n
            phase[s] ^= 1
            return s

        def first_bar():
            return (self.first[firsts % FIRST], firsts // FIRST & 1) if self.kept_first else (self.full[slot], phase[slot])

        def first_s(g, s, j, mine):
            qturn[g] += 1
            self.mma_s(g, s, j, 0)
            self.commit(self.s_full[g])
            if mine == 1:
                self.commit(self.q_empty[g])

        def next_s(g, s, j, i):
            self.mma_s(g, s, j, i)
            self.commit(self.s_full[g])

        ahead = False
        for j, nt in enumerate(self.items):
            if self.pair:
                for g in range(2):
                    if not nt[g]:
                        continue
                    yield first_bar()
                    yield self.q_full[g], qturn[g] & 1
                    firsts += 1
                    s = advance()
                    first_s(g, s, j, nt[g])
                    self.commit(self.empty[s])
                for i in range(max(nt)):
                    for g in range(2):
                        if i >= nt[g]:
                            continue
                        yield self.p_full[g], pturn[g] & 1
                        pturn[g] += 1
                        sv = advance()
                        self.mma_o(g, sv, j, i)
                        self.commit(self.o_done[g])
                        self.commit(self.empty[sv])
                        if i + 1 < nt[g]:
                            sk = advance()
                            next_s(g, sk, j, i + 1)
                            if i + 2 == nt[g]:
                                self.commit(self.q_empty[g])
                            self.commit(self.empty[sk])
                continue
            tiles = max(nt)
            next0 = self.items[j + 1][0] if j + 1 < len(self.items) else 0
            if not tiles:
                continue
            if not ahead:
                yield first_bar()
            firsts += 1
            s = advance()
            for g in range(2):
                if nt[g] and not (g == 0 and ahead):
                    yield self.q_full[g], qturn[g] & 1
                    first_s(g, s, j, nt[g])
            self.commit(self.empty[s])
            ahead = False
            for i in range(tiles):
                last = i + 1 == tiles
                sv, sk = advance(), None if last else advance()
                for g in range(2):
                    bar, parity = first_bar()
                    if last and g == 1 and i >= nt[0] and next0 and bar.done(parity) and \
                            self.q_full[0].done(qturn[0] & 1):
                        first_s(0, slot, j + 1, next0)
                        ahead = True
                    if i < nt[g]:
                        yield self.p_full[g], pturn[g] & 1
                        self.mma_o(g, sv, j, i)
                        pturn[g] += 1
                        self.commit(self.o_done[g])
                    if not last and i + 1 < nt[g]:
                        next_s(g, sk, j, i + 1)
                        if i + 2 == nt[g]:
                            self.commit(self.q_empty[g])
                self.commit(self.empty[sv])
                if not last:
                    self.commit(self.empty[sk])
        self.commit(self.drain)
        yield self.drain, 0

    def softmax(self, g, w):
        turn = 0
        for j, nt in enumerate(self.items):
            for i in range(nt[g]):
                yield self.s_full[g], turn & 1
                self.expect(self.s[g], (j, i), "S")
                yield None
                if i > 0 and self.rng.random() < 0.3:  # the reference is raised, O rescaled
                    yield self.o_done[g], (turn - 1) & 1
                    self.expect(self.o[g], [(j, x) for x in range(i)], "O while it grows")
                    yield None
                self.expect(self.s[g], (j, i), "S")
                self.p[g][w] = (j, i)
                self.p_full[g].arrive()
                turn += 1
                yield None
            if nt[g]:
                yield self.o_done[g], (turn - 1) & 1
                self.expect(self.o[g], [(j, x) for x in range(nt[g])], "O")
                yield None
                self.expect(self.o[g], [(j, x) for x in range(nt[g])], "O while it is read")
            self.written[j, g, w] = nt[g]

    def run(self):
        warps = [self.producer(), self.gate(), self.mma()] + [self.softmax(g, w) for g in range(2) for w in range(4)]
        waits = {k: None for k in range(len(warps))}
        # some runs hold one warp, the copies or the tensor cores back for long
        slow = self.rng.choice([None, "land", "pipe", *range(len(warps))])
        while True:
            able = [k for k, on in waits.items() if on is None or on[0].done(on[1])]
            able += ["land"] * bool(self.flying) + ["pipe"] * bool(self.pipe)
            if not able:
                break
            rest = [k for k in able if k != slow]
            k = self.rng.choice(rest if rest and self.rng.random() < 0.97 else able)
            if k == "land":
                self.land()
            elif k == "pipe":
                self.pipe.pop(0)()
            else:
                try:
                    waits[k] = next(warps[k])
                except StopIteration:
                    del waits[k]
        if waits:
            raise Wrong(f"warps {sorted(waits)} wait for ever")
        assert self.written == {(j, g, w): nt[g] for j, nt in enumerate(self.items) for g in range(2) for w in range(4)}


def some_items(rng, pair):
    """Key tiles of the two groups: short ones mostly, some long, groups without rows or keys among them."""
    items = []
    for _ in range(rng.randrange(1, 9)):
        a = rng.choice([0, 1, 1, 2, 2, 3, 5, 9])
        if pair:
            items.append((a, rng.choice([0, 1, 1, 2, 3, 7])))
        else:  # group 1 has the later queries: a key tile more at most, unless it has no rows
            items.append((a, rng.choice([0, a, a + 1]) if a else rng.choice([0, 1])))
    return items


@pytest.mark.parametrize("stages", [4, 8])   # head dim 128, 64
@pytest.mark.parametrize("pair", [False, True])
def test_every_read_finds_its_tile(stages, pair):
    for seed in range(400):
        rng = random.Random(seed)
        Cta(some_items(rng, pair), stages, pair, rng).run()


@pytest.mark.parametrize("stages", [4, 8])
def test_split_keys_are_a_single_item(stages):
    # the CTAs of a cluster take every ranks-th key tile: what one of them sees is a single item of any two lengths
    for seed in range(200):
        rng = random.Random(seed)
        a = rng.randrange(0, 12)
        Cta([(a, rng.choice([0, a, a + 1]))], stages, False, rng).run()


@pytest.mark.parametrize("stages,pair", [(4, False), (4, True), (8, True)])
def test_first_tiles_on_their_slots_barriers_are_caught(stages, pair):
    wrong = 0
    for seed in range(400):
        rng = random.Random(seed)
        try:
            Cta(some_items(rng, pair), stages, pair, rng, kept_first=False).run()
        except Wrong:
            wrong += 1
    assert wrong > 0
