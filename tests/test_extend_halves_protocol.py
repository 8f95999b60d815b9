"""The CPU model of test_extend_protocol.py for the kernel of capped bf16 scores, where two warps share their rows and have
half of the columns each: twice the softmax warps at every barrier that they arrive at, and exchanges of the halves' sums,
between the two warps of 32 rows or, where both query tiles are one, between all."""
import random

import pytest

from test_extend_protocol import RING, Bar, Model, items_of


class Halves(Model):
    def __init__(self, items, plant=""):
        super().__init__(items, False, plant)
        self.p_full = [Bar(4 if plant == "one half's arrivals" else 8) for _ in range(2)]
        self.item_empty = [Bar(16 + 3) for _ in range(RING)]
        self.xbar = Bar(16)
        self.rows = [[Bar(2) for _ in range(4)] for _ in range(2)]
        self.s = [[None] * 8 for _ in range(2)]                      # S / P per query tile, half and 32 rows
        self.red = [[[None, None] for _ in range(4)] for _ in range(2)]

    def tensor_core(self):
        for _ in super().tensor_core():
            for t in range(2):                                       # (a product writes both halves' columns)
                if len(self.s[t]) == 4:
                    self.s[t] = self.s[t] * 2
            yield

    def warp(self, t, half, quarter, rng):
        num = nx = nr = i = 0
        me = half * 4 + quarter

        def meet():
            nonlocal nx
            self.xbar.arrive()
            yield from self.wait(self.xbar, nx & 1)
            nx += 1

        def both(alt):
            nonlocal nr
            if alt:
                yield from meet()
                return
            bar = self.rows[t][quarter]
            bar.arrive()
            yield from self.wait(bar, nr & 1)
            nr += 1

        while True:
            w = yield from self.next_item(i)
            if w is None:
                return
            assert w["i"] == i
            alt, mine = w["alt"], []
            for j in range(w["n"][t]):
                jt = 2 * j + t if alt else j
                c = w["c0"] + jt
                st = (2 * c + 1) % self.nb
                yield from self.wait(self.s_full[t], num & 1)
                assert self.s[t][me] == ("s", c)
                if jt in w["edges"]:                                 # V's rows behind the context become 0
                    yield from self.wait(self.full[st], ((2 * c + 1) // self.nb) & 1)
                    self.reading[("kv", st)] = self.reading.get(("kv", st), 0) + 1
                    yield
                    assert self.kv[st] == 2 * c + 1
                    self.reading[("kv", st)] -= 1
                for _ in range(rng.choice([0, 2, 9])):
                    yield
                assert self.s[t][me] == ("s", c)
                self.s[t] = self.s[t][:me] + [("p", c)] + self.s[t][me + 1:]
                self.p_full[t].arrive()
                mine.append(c)
                num += 1
            if w["n"][t]:
                yield from self.wait(self.pv_done[t][(num - 1) & 1], ((num - 1) // 2) & 1)
                assert self.o[t] == mine
            # the halves' sums
            self.red[t][quarter][half] = ("sum", i, half)
            yield from both(alt)
            for u in (t, 1 - t) if alt else (t,):
                for _ in range(rng.choice([0, 3])):
                    yield
                assert self.red[u][quarter] == [("sum", i, 0), ("sum", i, 1)]
            if self.plant != "no second exchange":
                yield from both(alt)
            if alt:
                self.red[t][quarter][0] = ("max", i)                 # (the same in both halves)
                yield from meet()
                for _ in range(rng.choice([0, 3])):
                    yield
                assert self.red[1 - t][quarter][0] == ("max", i)
            read = [u for u in ((0, 1) if alt else (t,)) if w["n"][u]]
            for u in read:
                self.reading[("o", u)] = self.reading.get(("o", u), 0) + 1
            yield
            for u in read:
                assert self.o[u] == ([w["c0"] + 2 * k + u for k in range(w["n"][u])] if alt else mine)
                self.reading[("o", u)] -= 1
            if alt:
                yield from meet()
            if me == 0:
                self.out.append((i, t))
            self.item_empty[i % RING].arrive()
            i += 1

    def run(self, seed):
        rng = random.Random(seed)
        roles = [self.draw(), self.q_rows(), self.products(), self.v_copies()]
        roles += [self.warp(t, half, quarter, rng) for t in range(2) for half in range(2) for quarter in range(4)]
        core = self.tensor_core()
        slow = [rng.choice([1, 1, 1, 4, 60]) for _ in roles]
        live = list(range(len(roles)))
        for _ in range(3000000):
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


def test_random_schedules():
    for seed in range(40):
        rng = random.Random(seed)
        Halves(items_of(rng, rng.randint(1, 12))).run(seed)


def test_equal_tile_counts():
    """Tiles from the last one backwards (slopes) and spans: both query tiles take all of an item's KV tiles."""
    for seed in range(20):
        rng = random.Random(seed)
        items = [it if it[0] else (False, it[2], it[2], it[3]) for it in items_of(rng, 8)]
        Halves(items).run(seed)
        Model(items, seed % 2 == 0).run(seed)


@pytest.mark.parametrize("plant", ["one half's arrivals", "no second exchange"])
def test_planted_mistakes_are_caught(plant):
    for seed in range(20):
        rng = random.Random(seed)
        try:
            Halves(items_of(rng, 20), plant).run(seed)
        except AssertionError:
            return
    raise AssertionError("not caught")
