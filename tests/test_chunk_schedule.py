"""The chunk attention's hand-over between its warps (csrc/chunk_attn.cu), as a model: the roles
of a pair of CTAs as coroutines that run in a random order, every barrier with its counts, and
every buffer with what was last written to it. A wait is checked against the phase it means (the
hardware sees its parity only), a read against the contents it means.

The model takes the ring's sizes, whether a row's sums have an array of their own, and whether
the exponents of two items' queries have, from the kernel's source.

A wait that runs out aborts its CTA: none of its waits waits any more, nothing new is issued, and
its producer has to wait for what is still in flight before the CTA may exit."""

import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "decode_attention_10_b200", "csrc")
with open(os.path.join(CSRC, "chunk_attn.cu")) as _f:
    SOURCE = _f.read()
SLOTS, STAGE = (int(re.search(rf"constexpr int {name} = (\d+);", SOURCE).group(1))
                for name in ("kSlots", "kStageSlots"))
OWN_SUM = re.search(r"float sum\[2\]\[kRows\];", SOURCE) is not None
TWO_EXPONENTS = re.search(r"int32_t q_exp\[2\]\[kRows\];", SOURCE) is not None
NUMBERED = "bad_flag(" in SOURCE
ISSUED = "v_issued" in SOURCE and "q_issued" in SOURCE
QUADS = 2  # of the four: pairs of warps that share rows, in each CTA
WARPS = [(quad, half) for quad in range(QUADS) for half in range(2)]


class Fault(AssertionError):
    pass


def expect(ok, *what):
    if not ok and (Bar.strict or what[0] in ("hang", "in flight")):
        raise Fault(what)


class Bar:
    """An mbarrier: arrivals and outstanding bytes (in copies) of the current phase."""

    def __init__(self, name, count):
        self.name, self.count, self.left, self.tx, self.phase = name, count, count, 0, 0

    strict = True  # (not after an abort)

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase, self.left = self.phase + 1, self.count

    def arrive(self, tx=0):
        if self.left == 0 and not Bar.strict:
            return
        expect(self.left > 0, "too many arrivals", self.name, self.phase)
        self.tx += tx
        self.left -= 1
        self._turn()

    def complete(self):
        self.tx -= 1
        self._turn()

    def done(self, phase):
        """A wait for `phase`, which is at most the current one when it returns."""
        def ready():
            seen = (self.phase & 1) != (phase & 1)
            expect(seen == (self.phase > phase) or not Bar.strict, "parity", self.name, phase, self.phase)
            return seen
        ready.bar = self
        return ready


class Named:
    """A named barrier of `count` warps."""

    def __init__(self, count):
        self.count, self.here, self.turn = count, 0, 0

    def sync(self):
        mine = self.turn
        self.here += 1
        if self.here == self.count:
            self.here, self.turn = 0, self.turn + 1
        return lambda: self.turn > mine


class Model:
    """items: (blocks, the special ones of them, whole tile, tokens of the tile) each."""

    def __init__(self, seed, fp8, items, own_sum=OWN_SUM, two_exponents=TWO_EXPONENTS,
                 abort_at=None, numbered=NUMBERED, issued=ISSUED):
        self.rng = random.Random(seed)
        self.fp8, self.items, self.own_sum = fp8, items, own_sum
        self.two_exponents = two_exponents
        self.abort_at, self.abort = abort_at, [False, False]
        self.numbered, self.count_issued = numbered, issued
        self.ks = self.vs = 1 if fp8 else 2
        both, slots = range(2), range(SLOTS)
        warps = len(WARPS)
        self.kv_full = [Bar(("kv_full", s), 2) for s in slots]
        self.kv_empty = [[Bar(("kv_empty", r, s), 1) for s in slots] for r in both]
        self.v_full = [[Bar(("v_full", r, s), 1) for s in slots] for r in both]
        self.q_full = Bar("q_full", 2 if fp8 else 1)
        self.q_empty, self.stage_free, self.staged = (
            [Bar((name, r), count) for r in both]
            for name, count in (("q_empty", 1), ("stage_free", 1), ("staged", warps)))
        self.s_full, self.pv_done = ([[Bar((name, r, j), 1) for j in both] for r in both]
                                     for name in ("s_full", "pv_done"))
        self.p_full = [Bar(("p_full", j), 2 * warps) for j in both]
        self.o_free = Bar("o_free", 2 * warps)
        self.pair = [[Named(2) for _ in range(QUADS)] for _ in both]
        self.all = [Named(warps) for _ in both]
        self.late = [[Named(QUADS) for _ in both] for _ in both]  # (planted)
        # what each buffer holds
        self.ring = [[None] * SLOTS for _ in both]
        self.q = [[None] * warps for _ in both]
        self.q_exp = [[[None] * warps for _ in both] for _ in both]  # [CTA][item's parity][writer]
        self.xch, self.sum = ([[[None] * 2 for _ in range(QUADS)] for _ in both] for _ in both)
        self.bad = [[[0, 0], [0, 0]] for _ in both]  # [CTA][item's parity][V half]
        self.s_buf = [[[None] * warps for _ in both] for _ in both]  # [CTA][block's parity][warp]
        self.o = [None, None]
        self.copies = []  # landing in any order
        self.tensor = []  # done in order

    # blocks whose running maximum rises, and special blocks with a row held out: at random, the
    # same for all who ask
    def chance(self, share, *key):
        return random.Random(repr((self.items[0][0], *key))).random() < share

    def has_bad(self, half, k):
        return any(self.chance(.4, "bad", half, k, b) for b in sorted(self.items[k][1]))

    def copy(self, r, bar, what=None):
        """A copy of CTA r, which completes on `bar` in the phase that it has begun."""
        self.copies.append((bar, what, r, bar.phase))

    def load_q(self, r):
        if r == 0:
            self.q_full.arrive(tx=2)
        self.copy(r, self.q_full)

    def producer(self, r):
        at = specials = issued = v_issued = 0
        q_issued, abort = 1, self.abort

        def take():
            nonlocal at
            slot, use = at % SLOTS, at // SLOTS
            if use > 0:
                yield self.kv_empty[r][slot].done(use - 1)
            at += 1
            self.ring[r][slot] = None
            return slot

        def load_k(k, b):
            nonlocal issued
            for c in range(self.ks):
                slot = yield from take()
                if abort[r]:
                    continue
                self.kv_full[slot].arrive(tx=1)
                self.copy(r, self.kv_full[slot], (r, slot, ("K", k, b, c)))
                issued = at

        def load_v(k, b):
            nonlocal specials, issued, v_issued
            special, own = b in self.items[k][1], self.v_full[r][specials % SLOTS]
            for c in range(self.vs):
                slot = yield from take()
                if abort[r]:
                    continue
                if not special:
                    self.kv_full[slot].arrive(tx=1)
                elif c == 0:
                    own.arrive(tx=self.vs)
                if special:
                    v_issued = specials + 1
                self.copy(r, own if special else self.kv_full[slot], (r, slot, ("V", k, b, c)))
                issued = at
            specials += special

        for k, (n, _, whole, _) in enumerate(self.items):
            if not self.fp8 and k > 0:  # (the first item's by the helper)
                yield self.q_empty[r].done(k - 1)
                if not abort[r]:
                    self.load_q(r)
                    q_issued = k + 1
            yield from load_k(k, 0)
            for b in range(n):
                if b + 1 < n:
                    yield from load_k(k, b + 1)
                yield from load_v(k, b)
            if whole:
                for _ in range(STAGE):
                    slot = yield from take()
                    if not abort[r]:
                        self.kv_full[slot].arrive()
                if not abort[r]:
                    self.stage_free[r].arrive()
            yield None
        if not abort[r]:
            return
        # waits for the copies in flight: the last use of each barrier
        if not self.count_issued:  # (planted: counts what an abort has passed over too)
            v_issued, q_issued = specials, len(self.items)
        waits = [(self.v_full[r][c % SLOTS], c // SLOTS) for c in range(max(0, v_issued - SLOTS), v_issued)]
        if r == 0:
            waits += [(self.kv_full[c % SLOTS], c // SLOTS) for c in range(max(0, issued - SLOTS), issued)]
            if not self.fp8:
                waits.append((self.q_full, q_issued - 1))
        for bar, phase in waits:
            expect(bar.phase >= phase, "in flight", "a wait for nothing", bar.name, phase, bar.phase)
        # (the second CTA's on the first's barriers: given time to land)
        for bar, what, cta, phase in self.copies:
            expect(cta != r or (bar, phase) in waits or (r == 1 and bar.name not in [x.name for x in self.v_full[1]]),
                   "in flight", bar.name, what)
        self.copies = [x for x in self.copies if x[2] != r]

    def mma(self):
        at = t0 = 0

        def free(slot):
            return [self.kv_empty[r][slot].arrive for r in range(2)]

        def products(k, b, t):
            nonlocal at
            for c in range(self.ks):
                slot = at % SLOTS
                yield self.kv_full[slot].done(at // SLOTS)
                at += 1
                if self.abort[0]:
                    continue

                def work(slot=slot, c=c):
                    for r in range(2):
                        expect(self.ring[r][slot] == ("K", k, b, c), "K", self.ring[r][slot], k, b)
                        if self.fp8:
                            expect(self.q[r] == [k] * len(WARPS), "Q", self.q[r], k)
                        if c == self.ks - 1:
                            self.s_buf[r][t & 1] = [("S", t)] * len(WARPS)
                self.tensor.append([work, *free(slot)])
            if not self.abort[0]:
                self.tensor.append([self.s_full[r][t & 1].arrive for r in range(2)])

        def outputs(k, b, t):
            nonlocal at
            slots = []
            for _ in range(self.vs):
                slots.append(at % SLOTS)
                yield self.kv_full[at % SLOTS].done(at // SLOTS)
                at += 1
            if b == 0 and k > 0:
                yield self.o_free.done(k - 1)
            yield self.p_full[t & 1].done(t >> 1)
            if self.abort[0]:
                return
            for c, slot in enumerate(slots):
                def work(slot=slot, c=c):
                    for r in range(2):
                        expect(self.ring[r][slot] == ("V", k, b, c), "V", self.ring[r][slot], k, b)
                        expect(self.s_buf[r][t & 1] == [("P", t)] * len(WARPS), "P", k, b)
                        self.o[r] = (k, b)
                self.tensor.append([work, *free(slot)])
            self.tensor.append([self.pv_done[r][t & 1].arrive for r in range(2)])

        for k, (n, _, whole, _) in enumerate(self.items):
            yield self.q_full.done(k)
            yield from products(k, 0, t0)
            for b in range(n):
                if b + 1 < n:
                    yield from products(k, b + 1, t0 + b + 1)
                if b + 1 == n and not self.fp8 and not self.abort[0]:
                    self.tensor.append([self.q_empty[r].arrive for r in range(2)])
                if b + 1 == n and whole:
                    for c in range(STAGE):
                        x = at + self.vs + c
                        yield self.kv_full[x % SLOTS].done(x // SLOTS)
                yield from outputs(k, b, t0 + b)
            at += STAGE if whole else 0
            t0 += n

    def softmax(self, r, w):
        quad, half = WARPS[w]
        pair, t0, at, tiles = self.pair[r][quad], 0, 0, 0
        xch = self.xch[r][quad]
        sums = self.sum[r][quad] if self.own_sum else xch

        def next_q(k):
            exponents = self.q_exp[r][k & 1 if self.two_exponents else 0]
            self.q[r][w] = exponents[w] = k
            yield self.all[r].sync()
            if w == 0:
                self.q_full.arrive()
            yield None
            rows = exponents[2 * quad:2 * quad + 2]  # (the rows of a pair were split by two warps)
            expect(rows == [k, k], "exponent", k, rows)

        if self.fp8:
            yield from next_q(0)
        for k, (n, _, whole, tokens) in enumerate(self.items):
            real = 2 * r + quad < tokens
            for b in range(n):
                t = t0 + b
                yield self.s_full[r][t & 1].done(t >> 1)
                expect(self.s_buf[r][t & 1][w] == ("S", t), "S", k, b)
                if real:
                    yield pair.sync()
                    if b == 0 or self.chance(.4, "rise", r, quad, k, b):
                        xch[half] = ("max", k, b)
                        yield pair.sync()
                        yield None
                        expect(xch[half ^ 1] == ("max", k, b), "maximum", k, b, xch)
                        if b > 0:
                            yield self.pv_done[r][(t - 1) & 1].done((t - 1) >> 1)
                            expect(self.o[r] == (k, b - 1), "rescale", k, b)
                yield None
                self.s_buf[r][t & 1][w] = ("P", t)
                self.p_full[t & 1].arrive()
            t0 += n
            at += n * (self.ks + self.vs)
            if real:
                sums[half] = ("sum", k)
                yield pair.sync()
                yield None
                expect(sums[half ^ 1] == ("sum", k), "sum", k, sums)
            if self.fp8 and k + 1 < len(self.items):
                yield from next_q(k + 1)
            if whole:
                yield self.stage_free[r].done(tiles)
                tiles += 1
            yield self.pv_done[r][(t0 - 1) & 1].done((t0 - 1) >> 1)
            expect(self.o[r] == (k, n - 1), "result", k, self.o[r])
            bad = self.bad[r][k & 1][half]
            if self.numbered and bad != k + 1:
                bad = 0
            expect(bad == (k + 1 if self.has_bad(half, k) else 0), "flag", k, bad)
            yield None
            self.o_free.arrive()
            if whole:
                for c in range(2):
                    slot = (at + 2 * half + c) % SLOTS
                    held = self.ring[r][slot] or ("O", k, ())
                    expect(held[:2] == ("O", k), "stage", k, held)
                    if held[:2] == ("O", k):
                        self.ring[r][slot] = ("O", k, (*held[2], quad))
                at += STAGE
                yield None
                self.staged[r].arrive()
            if bad and not self.numbered:
                yield self.late[r][half].sync()
                if quad == 0:
                    self.bad[r][k & 1][half] = 0

    def helper(self, r):
        at = specials = tiles = 0
        for k, (n, special, whole, _) in enumerate(self.items):
            if not self.fp8 and k == 0:
                self.load_q(r)
            bad = False
            for b in sorted(special):
                v_at = at + self.ks + b * (self.ks + self.vs) + (self.ks if b + 1 < n else 0)
                yield self.v_full[r][specials % SLOTS].done(specials // SLOTS)
                specials += 1
                if self.abort[r]:
                    break
                bad |= self.chance(.4, "bad", r, k, b)
                if bad:
                    for x in range(2):
                        self.bad[x][k & 1][r] = k + 1
                for c in range(self.vs):
                    slot = (v_at + c) % SLOTS
                    expect(self.ring[r][slot] == ("V", k, b, c), "clean", self.ring[r][slot], k, b)
                    self.kv_full[slot].arrive()
                yield None
            at += n * (self.ks + self.vs)
            if whole:
                yield self.staged[r].done(tiles)
                tiles += 1
                if self.abort[r]:
                    continue
                for c in range(STAGE):
                    slot = (at + c) % SLOTS
                    held = self.ring[r][slot] or (None,)
                    expect(held[:2] == ("O", k) and sorted(held[2]) == list(range(QUADS)), "store", k, held)
                    yield None
                    self.kv_empty[r][slot].arrive()
                at += STAGE

    def run(self):
        Bar.strict = self.abort_at is None
        roles, cta = [self.mma()], [0]
        for r in range(2):
            roles += [self.producer(r), self.helper(r)]
            roles += [self.softmax(r, w) for w in range(len(WARPS))]
            cta += [r] * (2 + len(WARPS))
        waits = [None] * len(roles)
        weight = [self.rng.choice([1, 1, 5, 20]) for _ in roles]
        tensor, copies = (self.rng.choice([1, 5, 20]) for _ in range(2))
        alive = set(range(len(roles)))
        turn = 0
        while alive or self.tensor or self.copies:
            turn += 1
            if turn == self.abort_at:
                self.abort[self.rng.randrange(2)] = True
            ready = [i for i in sorted(alive)
                     if waits[i] is None or (self.abort[cta[i]] and hasattr(waits[i], "bar")) or waits[i]()]
            if not ready and not self.tensor and not self.copies and True in self.abort:
                expect(False in self.abort, "hang", self.items)
                self.abort[:] = [True, True]  # (the other CTA's waits run out as well)
                continue
            odds = [weight[i] for i in ready]
            if self.tensor:
                ready, odds = ready + ["tensor"], odds + [tensor]
            if self.copies:
                ready, odds = ready + ["copy"], odds + [copies]
            expect(ready, "all wait", self.items)
            which = self.rng.choices(ready, odds)[0]
            if which == "tensor":
                for step in self.tensor.pop(0):
                    step()
            elif which == "copy":
                bar, what, _, _ = self.copies.pop(self.rng.randrange(len(self.copies)))
                if what is not None:
                    self.ring[what[0]][what[1]] = what[2]
                bar.complete()
            else:
                try:
                    waits[which] = next(roles[which])
                except StopIteration:
                    alive.discard(which)


def random_items(rng):
    """A pair's items: whole tiles, of which the first and the last may be parts of tiles."""
    items, count = [], rng.randint(1, 7)
    for i in range(count):
        n = rng.choice([1, 1, 2, 3, 4, rng.randint(1, 12)])
        whole = 0 < i < count - 1 or rng.random() < .5
        hidden = rng.choice([1, 2]) if whole or i == 0 else rng.choice([0, 0, 1])
        items.append((n, frozenset(range(max(0, n - hidden), n)), whole, rng.randint(1, 4)))
    return items


def schedules(count, fp8, **layout):
    for seed in range(count):
        Model(seed, fp8, random_items(random.Random(seed)), **layout).run()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_every_wait_and_every_read_means_what_it_gets(fp8):
    schedules(250, fp8)


def test_the_model_sees_sums_that_overwrite_maxima():
    with pytest.raises(Fault, match="maximum"):
        schedules(250, False, own_sum=False)


def test_the_model_sees_one_array_of_exponents():
    with pytest.raises(Fault, match="exponent"):
        schedules(250, True, two_exponents=False)


def aborts(count, fp8, **layout):
    for seed in range(count):
        rng = random.Random(seed)
        items = random_items(rng)
        Model(seed, fp8, items, abort_at=rng.randint(1, 40 * sum(i[0] for i in items)), **layout).run()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_an_aborted_cta_waits_for_its_copies_in_flight(fp8):
    aborts(250, fp8)


def test_the_model_sees_flags_that_are_put_back_behind_a_barrier():
    # (after an abort some warps may see the flag and some not)
    with pytest.raises(Fault, match="hang"):
        aborts(1000, False, numbered=False)


def test_the_model_sees_waits_for_copies_that_were_not_issued():
    with pytest.raises(Fault, match="in flight"):
        aborts(250, False, issued=False)
