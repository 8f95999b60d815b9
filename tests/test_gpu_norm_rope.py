"""pa_norm_rope_reshape_and_cache against norms and complex multiplication in 64 bits, within bounds that count
roundings (scored_ref.NORM_STEPS)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import scored_ref
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64, to_bits

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


class Case:
    def __init__(self, seed, N, Hq, Hkv, D, bs, dtype, kv8=False, rot=None, axes=1, pairs=False, offset=0.0, weights=(True, True), far=5000, spread=1.0, eps=EPS):
        rng = np.random.default_rng(seed)
        self.N, self.Hq, self.Hkv, self.D, self.dtype, self.rot, self.pairs, self.axes, self.offset, self.eps = \
            N, Hq, Hkv, D, dtype, rot or D, pairs, axes, offset, eps
        n = self.rot // 2
        nb = -(-(N + 9) // bs)
        self.before = step_ref.Cache(nb, bs, Hkv, D, dtype, kv8, fill_nan=False)
        self.before.pool[:] = rng.integers(0, 200, self.before.pool.shape)      # what the call does not write stays
        size = lambda h: np.exp(rng.standard_normal((N, h, 1)) * spread)
        self.q, self.k = (to_bits(rng.standard_normal((N, h, D)) * size(h), dtype) for h in (Hq, Hkv))
        self.v = to_bits(rng.standard_normal((N, Hkv, D)), dtype)
        self.w = [to_bits(rng.standard_normal(D) * 0.3 + 1 - offset, dtype) if has else None for has in weights]
        self.slots = rng.permutation(nb * bs)[:N].astype(np.int64)
        self.pos = rng.integers(0, far, (axes, N)).astype(np.int32)
        self.pair_axis = (np.arange(n) * axes // n).astype(np.uint8)
        self.inv = 10000.0 ** (-np.arange(n) * 2 / self.rot)
        self.far = far
        ang = np.arange(far)[:, None] * self.inv
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)

    def weight(self, i):
        return None if self.w[i] is None else u16_to_dev(self.w[i], self.dtype)

    def run(self, in_place=False, with_q=True, err=None, stride=0):
        """(q_out bits, pool after)."""
        def rows(bits, extra):
            t = u16_to_dev(bits, self.dtype)
            if not extra:
                return t
            wide = torch.full((self.N, bits.shape[1] * self.D + extra), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :bits.shape[1] * self.D] = t.view(self.N, -1)
            return wide[:, :bits.shape[1] * self.D].unflatten(1, (bits.shape[1], self.D))
        c = self.before
        q, k, v = rows(self.q, stride), rows(self.k, stride * 2), rows(self.v, stride)
        q_out = q if in_place else torch.full((self.N, self.Hq, self.D), float("nan"), dtype=q.dtype, device="cuda")
        pool = torch.from_numpy(c.pool.view(np.int16) if not c.kv8 else c.pool.copy()).cuda()
        desc = pkv.CacheDesc(c.nb, c.bs, c.Hkv, c.D, step_ref.torch_dtype(self.dtype), kv_int8=c.kv8)
        pkv.norm_rope_reshape_and_cache(q_out if with_q else None, q if with_q else None, pool, desc, k, v, torch.from_numpy(self.slots).cuda(),
                                        torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.cos_sin).cuda(), self.weight(0), self.weight(1), self.eps,
                                        weight_offset=self.offset, pair_axis=self.pair_axis, interleaved=self.pairs, dev_err=err)
        after = step_ref.Cache(c.nb, c.bs, c.Hkv, c.D, c.dtype, c.kv8)
        got = pool.cpu().numpy()
        after.pool = got if c.kv8 else got.view(np.uint16)
        return dev_to_u16(q_out), after

    def turned(self, bits, i):
        """(64-bit result, bound on the fp32 errors before the result's own rounding)."""
        n = scored_ref.normed(bits_to_f64(bits, self.dtype), None if self.w[i] is None else bits_to_f64(self.w[i], self.dtype), self.offset, self.eps)
        ang = np.clip(self.pos, 0, self.far - 1)[self.pair_axis].T.astype(np.float64) * self.inv
        return step_ref.rotate64(n, ang, self.rot, self.pairs), scored_ref.NORM_STEPS * 2.0 ** -24 * scored_ref.pair_sizes(n, self.rot, self.pairs)

    def check(self, skipped=(), zero=(), **kw):
        q, after = self.run(**kw)
        u = step_ref.EPS[self.dtype] / 2
        tiny = 2.0 ** -25 if self.dtype == "f16" else 0.0
        if kw.get("with_q", True):
            want, tol = self.turned(self.q, 0)
            want[list(zero)] = 0
            assert (np.abs(bits_to_f64(q, self.dtype) - want) <= u * np.abs(want) * (1 + 2.0 ** -10) + tol + tiny).all()
            assert not q[list(zero)].any()
        c = self.before
        keep = np.setdiff1d(np.arange(self.N), np.asarray(skipped, int))
        block, t = self.slots[keep] // c.bs, self.slots[keep] % c.bs
        k, v = after.read(block, t, 0), after.read(block, t, 1)
        want, tol = self.turned(self.k, 1)
        want, tol, wv = want[keep], tol[keep], bits_to_f64(self.v, self.dtype)[keep]
        if c.kv8:
            # half a code step of the vector's largest element, its reciprocal and the scale a few fp32 steps off
            step = lambda x: np.abs(x).max(-1, keepdims=True) * (1 / 254 + 2.0 ** -20)
            assert (np.abs(k - want) <= step(want) + tol + tol.max(-1, keepdims=True)).all() and (np.abs(v - wv) <= step(wv)).all()
        else:
            assert (np.abs(k - want) <= u * np.abs(want) * (1 + 2.0 ** -10) + tol + tiny).all() and np.array_equal(v, wv)
        # nothing else is written
        blank = step_ref.Cache(c.nb, c.bs, c.Hkv, c.D, c.dtype, c.kv8)
        blank.pool = after.pool.copy()
        for cache in (blank, c):
            zeros = np.zeros((len(keep), c.Hkv, c.D), np.uint16)
            assert cache.write(zeros, zeros, self.slots[keep]) == 0
        assert np.array_equal(blank.pool, c.pool)
        return q, after


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("axes,rot,offset,weights", [(1, 0, 0.0, (True, True)), (3, 0, 1.0, (True, True)), (2, 48, 0.0, (True, False)), (1, 16, 1.0, (False, True)),
                                                     (4, 32, 0.0, (False, False))])
def test_results(pairs, D, kv8, dtype, axes, rot, offset, weights):
    Case(D + axes, 19, 6, 2, D, 8, dtype, kv8, rot, axes, pairs, offset, weights).check()


@pytest.mark.parametrize("bs", [1, 2, 4, 16, 32])
@pytest.mark.parametrize("kv8", [False, True])
def test_block_sizes(bs, kv8):
    Case(bs, 70, 3, 3, 128, bs, "bf16", kv8).check()


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 1, 1, 64), (1, 64, 8, 128), (2, 5, 1, 64), (607, 3, 1, 128), (613, 3, 1, 64), (2500, 5, 1, 128)])
def test_sizes(N, Hq, Hkv, D):
    Case(N, N, Hq, Hkv, D, 16, "bf16", axes=3).check()


def test_in_place_strided_and_without_queries():
    Case(1, 33, 4, 2, 128, 16, "f16").check(in_place=True)
    Case(2, 33, 4, 2, 64, 16, "bf16").check(stride=24)
    Case(3, 33, 4, 2, 128, 16, "bf16", kv8=True).check(with_q=False)


def test_length_does_not_matter():
    """A vector and its multiple by a power of two: the same bits where eps is nothing beside them."""
    c = Case(4, 30, 4, 2, 128, 16, "bf16", eps=1e-30)
    d = Case(4, 30, 4, 2, 128, 16, "bf16", eps=1e-30)
    for name in ("q", "k"):
        setattr(d, name, to_bits(bits_to_f64(getattr(c, name), "bf16") * 2.0 ** 20, "bf16"))
    (qa, a), (qb, b) = c.check(), d.check()
    assert np.array_equal(qa, qb) and np.array_equal(a.pool, b.pool)


def test_zero_small_and_large_vectors():
    """Zeros give zeros; vectors far below the root of eps are multiplied by about 1 / sqrt(eps); squares of large bf16
    vectors leave fp32, fp16's largest numbers do not."""
    for dtype, big in (("bf16", 3e38), ("f16", 65000.0)):
        c = Case(5, 12, 4, 2, 128, 16, dtype)
        rng = np.random.default_rng(6)
        for name, h in (("q", 4), ("k", 2)):
            x = getattr(c, name)
            x[0] = 0
            x[1] = to_bits(rng.uniform(-1, 1, (h, 128)) * (1e-30 if dtype == "bf16" else 1e-6), dtype)
            x[2] = to_bits(rng.uniform(-1, 1, (h, 128)) * big, dtype)
            x[3] = to_bits(np.full((h, 128), big), dtype)
            x[4, 0] = to_bits(rng.uniform(-1, 1, 128) * 2e19, dtype) if dtype == "bf16" else x[4, 0]
        q, _ = c.check()
        assert not (q[0] & 0x7FFF).any()                           # (zeros of either sign)


def test_vectors_that_are_not_finite():
    """NaN and infinities stay in their own vectors."""
    for kv8 in (False, True):
        c = Case(7, 8, 2, 2, 128, 16, "bf16", kv8)
        d = Case(7, 8, 2, 2, 128, 16, "bf16", kv8)
        for x in (d.q, d.k):
            x[1, 0, 5], x[2, 1, 70], x[3, 0, 0] = 0x7FC0, 0x7F80, 0xFF80
        (qa, a), (qb, b) = c.run(), d.run()
        bad = np.zeros((8, 2), bool)
        bad[1, 0] = bad[2, 1] = bad[3, 0] = True
        assert np.array_equal(qa[~bad], qb[~bad])
        assert np.isnan(bits_to_f64(qb[bad], "bf16")).any(-1).all()
        block, t = c.slots // 16, c.slots % 16
        ka, kb = a.read(block, t, 0), b.read(block, t, 0)
        assert np.array_equal(ka[~bad], kb[~bad])
        assert np.array_equal(a.read(block, t, 1), b.read(block, t, 1))


def test_skipped_and_bad_tokens():
    for kv8 in (False, True):
        c = Case(11, 24, 4, 2, 128, 16, "bf16", kv8, axes=3)
        c.slots[[2, 5]] = -1
        c.slots[7], c.slots[8] = c.before.nb * 16, -2
        c.pos[1, 9], c.pos[2, 10] = c.far, -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.check(skipped=[2, 5, 7, 8, 9, 10], zero=[9, 10], err=err)
        assert pkv.read_device_errors(err) == pkv.DEVERR_SLOT | pkv.DEVERR_POSITION


def test_agrees_with_the_call_without_norms():
    """Vectors of length sqrt(D) already, all of one size, eps small: what rope_reshape_and_cache gives, up to fp32 roundings of
    the norm (the mean is 1 up to 20 2^-24) and one step of the result's type."""
    c = Case(12, 40, 4, 2, 128, 16, "bf16", weights=(False, False), eps=1e-30)
    rng = np.random.default_rng(13)
    for name, h in (("q", 4), ("k", 2)):
        setattr(c, name, to_bits(rng.choice([-1.0, 1.0], (40, h, 128)), "bf16"))
    q, after = c.check()
    plain = torch.from_numpy(c.before.pool.view(np.int16).copy()).cuda()
    out = torch.empty(40, 4, 128, dtype=torch.bfloat16, device="cuda")
    pkv.rope_reshape_and_cache(out, u16_to_dev(c.q, "bf16"), plain, pkv.CacheDesc(c.before.nb, 16, 2, 128, torch.bfloat16), u16_to_dev(c.k, "bf16"),
                               u16_to_dev(c.v, "bf16"), torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.pos).cuda(), torch.from_numpy(c.cos_sin).cuda())
    a, b = bits_to_f64(q, "bf16"), out.double().cpu().numpy()
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 48 * 2.0 ** -24).all()


@pytest.mark.parametrize("kv8", [False, True])
def test_parts_of_one_row_in_place_and_a_layer(kv8):
    """q, k and v as slices of one projection's rows, q in place; a layer of a pool of three."""
    c = Case(16, 700, 4, 2, 128, 16, "bf16", kv8, axes=2)
    want = c.run()
    rows = torch.cat([u16_to_dev(b, "bf16").view(c.N, -1) for b in (c.q, c.k, c.v)], 1)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in rows.split([512, 256, 256], 1))
    b = c.before
    desc = pkv.CacheDesc(b.nb, 16, 2, 128, torch.bfloat16, num_layers=3, kv_int8=kv8)
    one = b.pool.view(np.uint8).reshape(-1)
    pool = torch.from_numpy(np.concatenate([one * 0, one, one * 0])).cuda()
    pkv.norm_rope_reshape_and_cache(q, q, pool, desc, k, v, torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.pos).cuda(),
                                    torch.from_numpy(c.cos_sin).cuda(), c.weight(0), c.weight(1), EPS, pair_axis=c.pair_axis, layer=1)
    assert np.array_equal(dev_to_u16(q), want[0])
    assert np.array_equal(dev_to_u16(k), c.k) and np.array_equal(dev_to_u16(v), c.v)
    got = pool.cpu().numpy().reshape(3, -1)
    assert np.array_equal(got[1], want[1].pool.view(np.uint8).reshape(-1)) and not got[0].any() and not got[2].any()


def test_weights_at_any_even_address():
    c = Case(18, 20, 4, 2, 128, 16, "f16")
    want = c.run()
    room = torch.zeros(300, dtype=torch.float16, device="cuda")
    room[1:129], room[131:259] = c.weight(0), c.weight(1)
    c.weight = lambda i: room[1:129] if i == 0 else room[131:259]
    got = c.run()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1].pool, want[1].pool)


def test_replays_on_another_stream_with_other_weights():
    """A captured call reads the weights, positions and slots of each replay."""
    c, d = Case(17, 90, 4, 2, 128, 16, "f16", axes=3), Case(19, 90, 4, 2, 128, 16, "f16", axes=3)
    want = [x.run() for x in (c, d)]
    desc = pkv.CacheDesc(c.before.nb, 16, 2, 128, torch.float16)
    state = lambda x: [u16_to_dev(b, "f16") for b in (x.q, x.k, x.v, x.w[0], x.w[1])] + [torch.from_numpy(a.copy()).cuda()
                                                                                        for a in (x.slots, x.pos, x.before.pool.view(np.int16))]
    t, cs = state(c), torch.from_numpy(c.cos_sin).cuda()
    out = torch.zeros_like(t[0])
    call = lambda: pkv.norm_rope_reshape_and_cache(out, t[0], t[7], desc, t[1], t[2], t[5], t[6], cs, t[3], t[4], EPS, pair_axis=c.pair_axis)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    for x, w in ((d, want[1]), (c, want[0])):
        for a, b in zip(t, state(x)):
            a.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(dev_to_u16(out), w[0]) and np.array_equal(t[7].cpu().numpy().view(np.uint16), w[1].pool)
