"""A CPU model of the chunk-attention kernel's barrier protocol (csrc/extend_tc.cu): its roles as coroutines
under random schedules, barriers with the hardware's parity semantics, and tags in place of data.  It checks
that every role finds the data it expects, that no buffer is overwritten while it is read, and that no
schedule deadlocks.  Mistakes planted in the model are caught."""
import random

import pytest

RING, SCALES = 4, 8


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def test(self, parity):                    # the phase of that parity has completed, as far as the parity tells
        return (self.phase & 1) != parity


class Model:
    """items: (alt, n0, n1, edge tiles) as the drawing warp publishes them."""

    def __init__(self, items, convert, plant=""):
        self.items, self.convert, self.plant = items, convert, plant
        fill = 4 if convert else 1
        self.nb = nb = 4 if convert else 5
        self.full, self.empty = [Bar(fill) for _ in range(nb)], [Bar(1) for _ in range(nb)]
        self.q_full, self.q_empty, self.s_full, self.p_full = [[Bar(4 if i == 3 else 1) for _ in range(2)] for i in range(4)]
        self.pv_done = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.item_full = [Bar(1) for _ in range(RING)]
        self.item_empty = [Bar(14 if convert else 11) for _ in range(RING)]
        self.xbar = Bar(8)
        self.work = [None] * RING
        self.kv, self.q = [None] * nb, [None] * 2
        self.sc = [[None] * 4 for _ in range(SCALES)]
        self.s = [[None] * 4 for _ in range(2)]          # S / P per query tile and warp
        self.o = [None] * 2
        self.reading = {}                                # (kind, index) -> readers
        self.tensor = []                                 # issued products and commits, executed in order
        self.out = []

    def wait(self, bar, parity):
        while not bar.test(parity):
            yield

    def tiles(self, w):
        return w["n"][0] + w["n"][1] if w["alt"] else max(w["n"])

    def draw(self):
        c = q0 = q1 = 0
        for i, it in enumerate(self.items + [None]):
            slot = i % RING
            if i >= RING:
                yield from self.wait(self.item_empty[slot], (i // RING - 1) & 1)
            if it is None:
                self.work[slot] = None
                self.item_full[slot].arrive()
                return
            alt, n0, n1, edges = it
            w = dict(i=i, alt=alt, n=(n0, n1), c0=c, qload=(q0, q1), edges=edges)
            q0 += n0 > 0
            q1 += (not alt) and n1 > 0
            self.work[slot] = w
            self.item_full[slot].arrive()
            n = self.tiles(w)
            if self.convert:
                c += n
                continue
            for j in range(n):
                yield from self.wait_empty(2 * c)
                yield
                self.fill(self.kv, "kv", 2 * c % self.nb, 2 * c)
                self.full[2 * c % self.nb].arrive()
                c += 1

    def fill(self, buf, kind, st, c):
        assert not self.reading.get((kind, st)), f"{kind} stage {st} overwritten while read"
        buf[st] = c

    def wait_empty(self, n):
        if n >= self.nb:
            yield from self.wait(self.empty[n % self.nb], (n // self.nb - 1) & 1)

    def next_item(self, i):
        yield from self.wait(self.item_full[i % RING], (i // RING) & 1)
        return self.work[i % RING]

    def v_copies(self):
        c = i = 0
        while True:
            w = yield from self.next_item(i)
            if w is None:
                return
            assert w["i"] == i
            for j in range(self.tiles(w)):
                yield from self.wait_empty(2 * c + 1)
                yield
                self.fill(self.kv, "kv", (2 * c + 1) % self.nb, 2 * c + 1)
                self.full[(2 * c + 1) % self.nb].arrive()
                c += 1
            self.item_empty[i % RING].arrive()
            i += 1

    def converter(self, me):
        c = i = 0
        while True:
            w = yield from self.next_item(i)
            if w is None:
                return
            for j in range(self.tiles(w)):
                yield from self.wait_empty(2 * c)
                yield
                n = SCALES
                assert not self.reading.get(("sc", c % n)), "scales overwritten while read"
                self.sc[c % n][me] = c
                for part in (0, 1):
                    if part:
                        yield from self.wait_empty(2 * c + 1)
                    yield
                    self.fill(self.kv, "kv", (2 * c + part) % self.nb, 2 * c + part)
                    self.full[(2 * c + part) % self.nb].arrive()
                c += 1
            self.item_empty[i % RING].arrive()
            i += 1

    def q_rows(self):
        i = 0
        while True:
            w = yield from self.next_item(i)
            if w is None:
                return
            for t in range(2):
                if w["n"][t] == 0 or (w["alt"] and t == 1):
                    continue
                load = w["qload"][t]
                if load > 0:
                    yield from self.wait(self.q_empty[t], (load - 1) & 1)
                yield
                self.fill(self.q, "q", t, i)
                self.q_full[t].arrive()
            self.item_empty[i % RING].arrive()
            i += 1

    def products(self):
        seen = {"k": 0, "v": 0, 0: 0, 1: 0}

        def filled(key, c):
            while seen[key] <= c:
                n = 2 * seen[key] + (key == "v")
                yield from self.wait(self.full[n % self.nb], (n // self.nb) & 1)
                seen[key] += 1

        def rows(t, load):
            while seen[t] <= load:
                yield from self.wait(self.q_full[t], seen[t] & 1)
                seen[t] += 1

        owed, num = [None, None], [0, 0]

        def pv(t):
            if owed[t] is None:
                return
            c, first, last = owed[t]
            yield from filled("v", c)
            yield from self.wait(self.p_full[t], num[t] & 1)
            self.tensor.append(("pv", t, (2 * c + 1) % self.nb, c, first))
            self.tensor.append(("commit", self.pv_done[t][num[t] & 1]))
            if last:
                self.tensor.append(("commit", self.empty[(2 * c + 1) % self.nb]))
            num[t] += 1
            owed[t] = None

        i = 0
        while True:
            slot = i % RING
            if not self.item_full[slot].test((i // RING) & 1):
                yield from pv(0)
                yield from pv(1)
                yield from self.wait(self.item_full[slot], (i // RING) & 1)
            w = self.work[slot]
            if w is None:
                yield from pv(0)
                yield from pv(1)
                return
            assert w["i"] == i
            self.item_empty[slot].arrive()
            alt, n = w["alt"], w["n"]
            yield from pv(0)
            if n[0] and seen[0] <= w["qload"][0] and not self.q_full[0].test(seen[0] & 1):
                yield from pv(1)
            for j in range(max(n)):
                for t in range(2):
                    yield
                    yield from pv(t)
                    if j >= n[t]:
                        continue
                    other = n[1 - t]
                    jt = 2 * j + t if alt else j
                    c = w["c0"] + jt
                    qt = 0 if alt else t
                    yield from filled("k", c)
                    yield from rows(qt, w["qload"][qt])
                    if jt in w["edges"]:
                        yield from filled("v", c)
                    last_k = alt or t == 1 or jt >= other or self.plant == "the first user releases"
                    last_q = j == n[t] - 1 and (not alt or (other < n[t] if t == 0 else other <= n[t]))
                    self.tensor.append(("qk", t, qt, 2 * c % self.nb, c, i))
                    self.tensor.append(("commit", self.s_full[t]))
                    if last_k:
                        self.tensor.append(("commit", self.empty[2 * c % self.nb]))
                    if last_q:
                        self.tensor.append(("commit", self.q_empty[qt]))
                    owed[t] = (c, j == 0, last_k)
            i += 1

    def tensor_core(self):
        while True:
            if not self.tensor:
                yield "idle"
                continue
            op = self.tensor[0]
            if op[0] == "commit":
                op[1].arrive()
            elif op[0] == "qk":
                _, t, qt, st, c, item = op
                for key in (("kv", st), ("q", qt)):
                    self.reading[key] = self.reading.get(key, 0) + 1
                yield
                assert self.kv[st] == 2 * c and self.q[qt] == item, (self.kv, self.q, op)
                for key in (("kv", st), ("q", qt)):
                    self.reading[key] -= 1
                self.s[t] = [("s", c)] * 4
            else:
                _, t, st, c, first = op
                self.reading[("kv", st)] = self.reading.get(("kv", st), 0) + 1
                yield
                assert self.kv[st] == 2 * c + 1 and all(x == ("p", c) for x in self.s[t]), op
                self.reading[("kv", st)] -= 1
                assert not self.reading.get(("o", t)), "accumulator overwritten while read"
                self.o[t] = [c] if first else self.o[t] + [c]
            self.tensor.pop(0)
            yield

    def softmax(self, t, me, rng):
        num = nx = i = 0
        while True:
            w = yield from self.next_item(i)
            if w is None:
                return
            assert w["i"] == i
            mine = []
            for j in range(w["n"][t]):
                jt = 2 * j + t if w["alt"] else j
                c = w["c0"] + jt
                st = (2 * c + 1) % self.nb
                yield from self.wait(self.s_full[t], num & 1)
                assert self.s[t][me] == ("s", c)
                if self.convert:
                    n = SCALES
                    self.reading[("sc", c % n)] = self.reading.get(("sc", c % n), 0) + 1
                    assert self.sc[c % n] == [c] * 4
                    for _ in range(rng.choice([0, 1, 30])):
                        yield
                    assert self.sc[c % n] == [c] * 4
                    self.reading[("sc", c % n)] -= 1
                if jt in w["edges"] and not self.convert:
                    yield from self.wait(self.full[st], ((2 * c + 1) // self.nb) & 1)
                    self.reading[("kv", st)] = self.reading.get(("kv", st), 0) + 1
                    yield
                    assert self.kv[st] == 2 * c + 1
                    self.reading[("kv", st)] -= 1
                if j > 0 and rng.random() < 0.3:         # the rescale
                    yield from self.wait(self.pv_done[t][(num - 1) & 1], ((num - 1) // 2) & 1)
                    assert self.o[t][-1] == c - (2 if w["alt"] else 1)
                for _ in range(rng.choice([0, 2, 9])):
                    yield
                self.s[t] = self.s[t][:me] + [("p", c)] + self.s[t][me + 1:]
                self.p_full[t].arrive()
                mine.append(c)
                num += 1
            if w["n"][t]:
                yield from self.wait(self.pv_done[t][(num - 1) & 1], ((num - 1) // 2) & 1)
                assert self.o[t] == mine
            if w["alt"]:
                self.xbar.arrive()
                yield from self.wait(self.xbar, nx & 1)
                nx += 1
                for u in range(2):
                    if w["n"][u]:
                        self.reading[("o", u)] = self.reading.get(("o", u), 0) + 1
                yield
                for u in range(2):
                    if w["n"][u]:
                        assert self.o[u] == [w["c0"] + 2 * k + u for k in range(w["n"][u])]
                        self.reading[("o", u)] -= 1
                if self.plant != "no second meeting":
                    self.xbar.arrive()
                    yield from self.wait(self.xbar, nx & 1)
                    nx += 1
            if me == 0:
                self.out.append((i, t))
            self.item_empty[i % RING].arrive()
            i += 1

    def run(self, seed):
        rng = random.Random(seed)
        roles = [self.draw(), self.q_rows(), self.products()]
        roles += [self.converter(m) for m in range(4)] if self.convert else [self.v_copies()]
        roles += [self.softmax(t, m, rng) for t in range(2) for m in range(4)]
        core = self.tensor_core()
        slow = [rng.choice([1, 1, 1, 4, 60]) for _ in roles]
        live = list(range(len(roles)))
        for step in range(3000000):
            if not live:
                break
            r = rng.randrange(len(roles) + 2)
            if r >= len(roles):
                next(core)
            elif r in live and rng.randrange(slow[r]) == 0:
                try:
                    next(roles[r])
                except StopIteration:
                    live.remove(r)
        assert not live, "deadlock"
        assert sorted(self.out) == [(i, t) for i in range(len(self.items)) for t in range(2)]


def items_of(rng, count):
    items = []
    for _ in range(count):
        if rng.random() < 0.5:
            n = rng.choice([0, 1, 1, 1, 2, 3, 5])
            items.append((True, (n + 1) // 2, n // 2, set(rng.sample(range(n), min(n, rng.randint(0, 2))))))
        else:
            n = rng.choice([1, 1, 2, 3])
            n0 = n - rng.randint(0, 1)
            items.append((False, n0, n, set(rng.sample(range(n), rng.randint(0, min(n, 2))))))
    return items


@pytest.mark.parametrize("convert", [False, True])
def test_random_schedules(convert):
    for seed in range(60):
        rng = random.Random(seed)
        Model(items_of(rng, rng.randint(1, 12)), convert).run(seed)


@pytest.mark.parametrize("convert", [False, True])
@pytest.mark.parametrize("plant", ["no second meeting", "the first user releases"])
def test_planted_mistakes_are_caught(plant, convert):
    for seed in range(20):
        rng = random.Random(seed)
        try:
            Model(items_of(rng, 20), convert, plant).run(seed)
        except AssertionError:
            return
    raise AssertionError("not caught")
