"""pa_build_tables against the plain reference: every output equal, number by number."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x).astype(dtype)).cuda()


class Step:
    def __init__(self, seed, cached, new, bs, ring=0, width=None, spare=4, pad=0, num_blocks=None):
        rng = np.random.default_rng(seed)
        self.cached, self.new, self.bs, self.ring = np.asarray(cached, np.int32), np.asarray(new, np.int32), bs, ring
        S = len(self.cached)
        blocks = lambda x: np.minimum(-(-x.astype(np.int64) // bs), ring or 1 << 40)
        have, need = blocks(np.maximum(self.cached, 0)), blocks(np.maximum(self.cached + self.new, 0))
        self.width = width or ring or max(int(need.max(initial=1)), 1)
        self.nb = num_blocks or int(need.sum()) + spare
        perm = rng.permutation(self.nb).astype(np.int32)
        self.tables = np.full((S, self.width), -7, np.int32)
        at = 0
        for s in range(S):
            n = min(int(have[s]), self.width)
            self.tables[s, :n] = perm[at:at + n]
            at += n
        self.num_free = self.nb - at
        self.free = np.full(self.nb, -9, np.int32)
        self.free[:self.num_free] = perm[at:]
        self.max_tokens = int(np.maximum(self.new, 0).sum()) + pad

    def check(self, want_err=0, in_place=False, positions=True, stream=None):
        t = dict(tables=dev(self.tables), free=dev(self.free), nf=dev([self.num_free]), cached=dev(self.cached), new=dev(self.new))
        S = len(self.cached)
        # guards behind every output
        qsl, ctx = dev(np.full(S + 3, 77)), t["cached"] if in_place else dev(np.full(S + 2, 77))
        slots, pos = dev(np.full(self.max_tokens + 2, 77), np.int64), dev(np.full(self.max_tokens + 2, 77))
        nfo = t["nf"] if in_place else dev([77])
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        desc = pkv.CacheDesc(self.nb, self.bs, 1, 128)
        pkv.build_tables(qsl[:S + 1], ctx[:S], slots[:self.max_tokens], pos[:self.max_tokens] if positions else None, t["tables"],
                         t["free"], t["nf"], nfo, desc, t["cached"], t["new"], ring_blocks=self.ring, dev_err=err)
        bits = pkv.read_device_errors(err)
        want = step_ref.build_tables(self.tables, self.free, self.num_free, self.cached, self.new, self.nb, self.bs, self.ring,
                                     self.max_tokens)
        assert bits == want[6] == want_err
        assert np.array_equal(qsl[:S + 1].cpu().numpy(), want[0])
        assert np.array_equal(ctx[:S].cpu().numpy(), want[1])
        assert np.array_equal(slots[:self.max_tokens].cpu().numpy(), want[2])
        if positions:
            assert np.array_equal(pos[:self.max_tokens].cpu().numpy(), want[3])
        assert np.array_equal(t["tables"].cpu().numpy(), want[4])
        assert nfo.item() == want[5]
        assert np.array_equal(t["free"].cpu().numpy(), self.free)
        assert (qsl[S + 1:] == 77).all() and (slots[self.max_tokens:] == 77).all() and (pos[self.max_tokens:] == 77).all()
        if not in_place:
            assert (ctx[S:] == 77).all()


@pytest.mark.parametrize("bs", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("ring", [0, 3])
@pytest.mark.parametrize("pad", [0, 37])
def test_mixed_lengths(bs, ring, pad):
    rng = np.random.default_rng(bs * 10 + ring)
    cached = np.concatenate([[0, 0, 1, bs, bs - 1, bs + 1, 5 * bs], rng.integers(0, 9 * bs, 40)])
    new = np.concatenate([[0, 1, 0, 1, 1, bs, 7 * bs + 1], rng.integers(0, 6 * bs, 40)])
    Step(bs, cached, new, bs, ring, pad=pad).check()


@pytest.mark.parametrize("S,hi", [(1, 1), (1, 5000), (31, 1), (1024, 3), (1025, 2), (4096, 3), (16384, 1)])
def test_sizes(S, hi):
    rng = np.random.default_rng(S)
    Step(S, rng.integers(0, 40, S), rng.integers(0, hi + 1, S), 16, pad=5).check()


def test_long_prompts_and_a_wide_table():
    Step(5, [0, 100, 0], [9000, 20000, 1], 16, width=2000, pad=1).check()


def test_nothing_new_and_no_requests():
    Step(6, [5, 17, 0], [0, 0, 0], 16, pad=3).check()
    Step(7, [], [], 16, pad=4, num_blocks=4).check()


@pytest.mark.parametrize("ring", [0, 4])
def test_update_in_place(ring):
    Step(8, [3, 0, 100, 16], [5, 40, 1, 0], 8, ring).check(in_place=True)


def test_without_positions():
    Step(9, [3, 0], [5, 40], 8, pad=2).check(positions=False)


def test_exactly_enough_blocks():
    Step(10, [0, 15], [33, 2], 16, spare=0).check()


def test_steps_that_cannot_be_built_are_empty():
    s = Step(11, [0, 15, 40], [33, 2, 1], 16)
    s.num_free = 2                                                  # needs four
    s.check(want_err=32)
    for bad in (-1, s.nb + 1):
        s.num_free = bad
        s.check(want_err=32)
    s = Step(12, [0, -1, 40], [33, 2, 1], 16)
    s.check(want_err=4)                                             # a negative length
    s = Step(13, [0, 9], [33, -2], 16)
    s.check(want_err=4)
    s = Step(14, [0, 60], [20, 9], 16, width=4)
    s.check(want_err=4)                                             # past its row
    s = Step(15, [0, 2**31 - 2], [1, 2], 16, ring=4)
    s.check(want_err=4)                                             # past int32
    s = Step(16, [0, 5], [33, 2], 16)
    s.max_tokens -= 1
    s.check(want_err=4)                                             # more tokens than rows
    s = Step(17, [0, 2**31 - 1], [2**31 - 1, 0], 16, ring=4, num_blocks=20)
    s.max_tokens = 50
    s.check(want_err=4)                                             # sums past int32


def test_bad_block_ids_skip_their_tokens():
    s = Step(18, [0, 15, 40], [33, 2, 1], 16)
    s.free[s.num_free - 2] = s.nb                                   # the first request's second block
    s.tables[2, 2] = -1                                             # the third one's last block
    s.check(want_err=1)


def test_long_contexts_in_a_ring():
    # positions near 2^31, slots past 2^31 are out of a table's reach: ids are int32, blocks up to 32 tokens
    s = Step(19, [2**31 - 60], [59], 32, ring=3)
    s.check()


def test_captured_step_follows_its_lengths():
    """One captured call, replayed with other lengths in the same buffers."""
    s = Step(20, [10, 0, 33], [1, 20, 3], 16, pad=40, spare=30)
    other = Step(20, [10, 0, 33], [9, 2, 30], 16, spare=30)
    other.nb, other.width = s.nb, max(s.width, other.width)
    S, T = 3, s.max_tokens
    tables = np.full((S, other.width), -7, np.int32)
    tables[:, :s.width] = s.tables
    bufs = dict(qsl=dev(np.zeros(S + 1)), ctx=dev(np.zeros(S)), slots=dev(np.zeros(T), np.int64), pos=dev(np.zeros(T)),
                tables=dev(tables), free=dev(s.free), nf=dev([s.num_free]), nfo=dev([0]), cached=dev(s.cached), new=dev(s.new))
    desc = pkv.CacheDesc(s.nb, 16, 1, 128)
    call = lambda: pkv.build_tables(bufs["qsl"], bufs["ctx"], bufs["slots"], bufs["pos"], bufs["tables"], bufs["free"], bufs["nf"],
                                    bufs["nfo"], desc, bufs["cached"], bufs["new"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    for new in (s.new, other.new, s.new):
        bufs["tables"].copy_(dev(tables))
        bufs["new"].copy_(dev(new))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step_ref.build_tables(tables, s.free, s.num_free, s.cached, new, s.nb, 16, 0, T)
        for k, w in zip(("qsl", "ctx", "slots", "pos", "tables"), want):
            assert np.array_equal(bufs[k].cpu().numpy(), w), k
        assert bufs["nfo"].item() == want[5]


@pytest.mark.parametrize("ring", [0, 4])
def test_a_failed_update_in_place_can_be_tried_again(ring):
    """Too few blocks, in place: lengths, tables and the free list stay as they were; with more blocks the same
    call builds the step."""
    s = Step(21, [30, 0, 17, 9], [20, 40, 1, 0], 8, ring)
    S, T = 4, s.max_tokens
    free = s.free.copy()
    z = lambda *n, dt=torch.int32: torch.full(n, 77, dtype=dt, device="cuda")
    qsl, slots, pos, err = z(S + 1), z(T, dt=torch.int64), z(T), z(1) * 0
    tables, lens, new, nf = dev(s.tables), dev(s.cached), dev(s.new), dev([2])
    desc = pkv.CacheDesc(s.nb, 8, 1, 128)
    call = lambda: pkv.build_tables(qsl, lens, slots, pos, tables, dev(free), nf, nf, desc, lens, new, ring_blocks=ring, dev_err=err)
    call()
    assert pkv.read_device_errors(err) == pkv.DEVERR_OUT_OF_BLOCKS
    assert lens.tolist() == s.cached.tolist() and nf.item() == 2
    assert np.array_equal(tables.cpu().numpy(), s.tables)
    assert not qsl.any() and bool((slots == -1).all()) and not pos.any()
    nf.fill_(s.num_free)
    call()
    assert pkv.read_device_errors(err) == 0
    want = step_ref.build_tables(s.tables, free, s.num_free, s.cached, s.new, s.nb, 8, ring, T)
    for got, w in zip((qsl, lens, slots, pos, tables), want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert nf.item() == want[5]
    # any other reason for an empty step leaves them as well
    lens, new = dev([30, -1, 17, 9]), dev([1, 1, 1, 1])
    call()
    assert pkv.read_device_errors(err) & pkv.DEVERR_CONTEXT
    assert lens.tolist() == [30, -1, 17, 9]


def test_tables_that_are_part_of_wider_rows():
    """A view of the first entries of longer rows: contexts are held to its width, and what lies behind it stays."""
    s = Step(22, [30, 0, 17], [20, 40, 1], 8, width=7)
    S, T = 3, s.max_tokens
    wide = dev(np.concatenate([s.tables, np.full((S, 5), 55)], 1))
    z = lambda *n, dt=torch.int32: torch.full(n, 77, dtype=dt, device="cuda")
    qsl, ctx, slots, pos, nfo, err = z(S + 1), z(S), z(T, dt=torch.int64), z(T), z(1), z(1) * 0
    desc = pkv.CacheDesc(s.nb, 8, 1, 128)

    def call(new, ring=0):
        pkv.build_tables(qsl, ctx, slots, pos, wide[:, :7], dev(s.free), dev([s.num_free]), nfo, desc, dev(s.cached), dev(new), ring_blocks=ring, dev_err=err)
    call(np.asarray([27, 40, 1]))                                    # 57 tokens: eight blocks
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((wide[:, 7:] == 55).all()) and np.array_equal(wide[:, :7].cpu().numpy(), s.tables) and not qsl.any()
    with pytest.raises(pkv.PagedKVError):
        call(s.new, ring=8)
    call(s.new)
    assert pkv.read_device_errors(err) == 0
    want = step_ref.build_tables(s.tables, s.free, s.num_free, s.cached, s.new, s.nb, 8, 0, T)
    for got, w in zip((qsl, ctx, slots, pos, wide[:, :7], nfo), want):
        assert np.array_equal(got.cpu().numpy(), np.atleast_1d(w))
    assert bool((wide[:, 7:] == 55).all())
