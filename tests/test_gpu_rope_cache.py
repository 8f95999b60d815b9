"""pa_rope_reshape_and_cache: bit for bit against binary32 arithmetic and the oracle's cache layout, and
against complex multiplication in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64, to_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


class Case:
    def __init__(self, seed, N, Hq, Hkv, D, bs, dtype, kv8=False, rot=None, axes=1, pairs=False, cycle=False, far=5000, base=10000.0):
        rng = np.random.default_rng(seed)
        self.N, self.Hq, self.Hkv, self.D, self.dtype, self.rot, self.pairs, self.axes = N, Hq, Hkv, D, dtype, rot or D, pairs, axes
        n = self.rot // 2
        nb = -(-(N + 9) // bs)
        self.before = step_ref.Cache(nb, bs, Hkv, D, dtype, kv8, fill_nan=False)
        self.before.pool[:] = rng.integers(0, 200, self.before.pool.shape)      # what the call does not write stays
        self.q, self.k, self.v = (to_bits(rng.standard_normal((N, h, D)) * 2, dtype) for h in (Hq, Hkv, Hkv))
        self.slots = rng.permutation(nb * bs)[:N].astype(np.int64)
        self.pos = rng.integers(0, far, (axes, N)).astype(np.int32)
        self.pos[:, rng.integers(0, N)] = far - 1
        self.pair_axis = (np.arange(n) % axes if cycle else np.arange(n) * axes // n).astype(np.uint8)
        self.inv = base ** (-np.arange(n) * 2 / self.rot)
        self.far = far
        ang = np.arange(far)[:, None] * self.inv
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)

    def run(self, in_place=False, with_q=True, err=None, stride=0, no_axes=False):
        """(q_out bits, pool)."""
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
        pos = torch.from_numpy(self.pos[0] if no_axes else self.pos).cuda()
        pkv.rope_reshape_and_cache(q_out if with_q else None, q if with_q else None, pool, desc, k, v, torch.from_numpy(self.slots).cuda(), pos,
                                   torch.from_numpy(self.cos_sin).cuda(), pair_axis=None if no_axes else self.pair_axis, interleaved=self.pairs,
                                   dev_err=err)
        torch.cuda.synchronize()
        pool = pool.cpu().numpy()
        return dev_to_u16(q_out), pool if c.kv8 else pool.view(np.uint16)

    def expected(self):
        """Binary32 results: (q bits, pool)."""
        ok = ((self.pos >= 0) & (self.pos < self.far))[np.unique(self.pair_axis)].all(0)
        pos = np.where(ok[None], self.pos, 0)
        n = self.rot // 2
        row = self.cos_sin[pos[self.pair_axis].T]                               # [N, n, rot]
        cos, sin = row[:, np.arange(n), np.arange(n)], row[:, np.arange(n), np.arange(n) + n]
        f = lambda bits: bits_to_f64(bits, self.dtype).astype(np.float32)
        turn = lambda bits: step_ref.rotate32(f(bits), cos, sin, self.rot, self.pairs)
        q = to_bits(turn(self.q), self.dtype)
        q[~ok] = 0
        c = self.before
        after = step_ref.Cache(c.nb, c.bs, c.Hkv, c.D, c.dtype, c.kv8)
        after.pool = c.pool.copy()
        slots = np.where(ok & (self.slots >= 0) & (self.slots < c.nb * c.bs), self.slots, -1)
        if c.kv8:
            for part, x in enumerate((turn(self.k), f(self.v))):
                step_ref.store8(after, *step_ref.quantise(x), part, slots)
        else:
            assert after.write(to_bits(turn(self.k), self.dtype), self.v, slots) == 0
        return q, after.pool

    def check(self, **kw):
        got, want = self.run(**kw), self.expected()
        if kw.get("with_q", True):
            assert np.array_equal(got[0], want[0])
        assert np.array_equal(got[1], want[1])
        return got


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("axes,cycle,rot", [(1, False, 0), (3, False, 0), (3, True, 32), (2, True, 48), (4, False, 16)])
def test_bits(pairs, D, kv8, dtype, axes, cycle, rot):
    Case(D + axes, 19, 6, 2, D, 8, dtype, kv8, rot, axes, pairs, cycle).check()


@pytest.mark.parametrize("bs", [1, 2, 4, 16, 32])
@pytest.mark.parametrize("kv8", [False, True])
def test_block_sizes(bs, kv8):
    Case(bs, 70, 3, 3, 128, bs, "bf16", kv8).check()


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (1, 64, 8), (2, 5, 1), (1300, 8, 2), (2500, 2, 1)])
def test_sizes(N, Hq, Hkv):
    Case(N, N, Hq, Hkv, 128, 16, "bf16", axes=3).check()


def test_in_place_strided_without_queries_and_without_axes():
    Case(1, 33, 4, 2, 128, 16, "f16").check(in_place=True)
    Case(2, 33, 4, 2, 64, 16, "bf16").check(stride=24)
    Case(3, 33, 4, 2, 128, 16, "bf16", kv8=True).check(with_q=False)
    Case(4, 33, 4, 2, 128, 16, "bf16").check(no_axes=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_against_complex_multiplication_in_64_bits(dtype, pairs):
    """Far positions, two axes.  Each result is off by the output's rounding (half a step), and by cos and
    sin rounded to fp32 (2^-24 each) and three fp32 roundings: 5 * 2^-24 (|x1| + |x2|)."""
    c = Case(7, 40, 4, 2, 128, 16, dtype, axes=2, pairs=pairs, cycle=True, far=131072)
    q, _ = c.check()
    ang = c.pos[c.pair_axis].T.astype(np.float64) * c.inv
    x = bits_to_f64(c.q, dtype)
    want = step_ref.rotate64(x, ang, 128, pairs)
    size = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]) if pairs else np.abs(x[..., :64]) + np.abs(x[..., 64:])
    size = np.repeat(size, 2, -1) if pairs else np.concatenate([size, size], -1)
    tol = step_ref.EPS[dtype] / 2 * np.abs(want) + 6 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "f16" else 0)
    assert (np.abs(bits_to_f64(q, dtype) - want) <= tol).all()


def test_scores_depend_on_distance_only():
    """q at position a against k at position b: the same product for every pair of positions b = a + 5, up to
    the rounding of the stored vectors (bf16: half a step of each element, both sides)."""
    N = 50
    c = Case(9, N, 1, 1, 128, 16, "bf16", far=4000)
    c.q[:], c.k[:] = c.q[:1], c.k[:1]
    c.pos[0] = np.arange(N) * 70
    q, _ = c.run()
    d = Case(9, N, 1, 1, 128, 16, "bf16", far=4000)
    d.q[:], d.pos[0] = c.k[:1], c.pos[0] + 5                                    # the key as a query, to read it back
    k, _ = d.run()
    a, b = bits_to_f64(q, "bf16")[:, 0], bits_to_f64(k, "bf16")[:, 0]
    z = (a * b).sum(-1)
    bound = 2 * (2.0 ** -8 * 2.01) * np.sqrt((a * a).sum(-1) * (b * b).sum(-1))
    assert (np.abs(z - z[0]) <= bound).all()


@pytest.mark.parametrize("size", [1e-37, 1e-38, 1e-40])
def test_codes_of_vectors_near_the_smallest_numbers(size):
    """127 / max|x| leaves fp32's range."""
    case = Case(77, 20, 2, 2, 128, 16, "bf16", kv8=True)
    rng = np.random.default_rng(78)
    case.k, case.v = (to_bits(rng.uniform(-1, 1, (20, 2, 128)) * size, "bf16") for _ in range(2))
    got, want = case.run(), case.expected()
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


def test_skipped_and_bad_tokens():
    for kv8 in (False, True):
        c = Case(11, 24, 4, 2, 128, 16, "bf16", kv8, axes=3)
        c.slots[[2, 5]] = -1
        c.slots[7], c.slots[8] = c.before.nb * 16, -2
        c.pos[1, 9], c.pos[2, 10] = c.far, -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.check(err=err)
        assert pkv.read_device_errors(err) == pkv.DEVERR_SLOT | pkv.DEVERR_POSITION


def test_a_bad_position_of_an_unused_axis_does_not_matter():
    c = Case(12, 10, 2, 1, 64, 8, "f16", axes=2)
    c.pair_axis[:] = 0
    c.pos[1] = -5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(err=err)
    assert pkv.read_device_errors(err) == 0


def test_special_values_pass_through():
    """Zero vectors store scale 0; infinities and NaN of v are stored as they are (16-bit)."""
    c = Case(13, 6, 2, 2, 128, 8, "bf16")
    c.v[0, 0, :4] = [0x7F80, 0xFF80, 0x7FC0, 0x8000]
    c.check()
    c = Case(14, 6, 2, 2, 128, 8, "bf16", kv8=True)
    c.k[1], c.v[2] = 0, 0
    c.check()


def test_long_cache_offsets():
    """Slots whose byte offset passes 2^32 (a pool of 5 GB)."""
    c = Case(15, 8, 2, 8, 128, 16, "bf16")
    nb = 5 * 2**30 // (8 * 2 * 16 * 128 * 2)
    pool = torch.zeros(nb * 8 * 2 * 16 * 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(8, dtype=torch.int64, device="cuda") + (nb - 1) * 16
    desc = pkv.CacheDesc(nb, 16, 8, 128, torch.bfloat16)
    k, v = u16_to_dev(c.k, "bf16"), u16_to_dev(c.v, "bf16")
    pkv.rope_reshape_and_cache(None, None, pool, desc, k, v, slots, torch.from_numpy(c.pos[0]).cuda(), torch.from_numpy(c.cos_sin).cuda())
    last = dev_to_u16(pool[-8 * 2 * 16 * 128:])
    c.before = step_ref.Cache(1, 16, 8, 128, "bf16", False, fill_nan=False)
    c.slots = np.arange(8)
    assert np.array_equal(last, c.expected()[1])
    assert int(pool[:-8 * 2 * 16 * 128].count_nonzero()) == 0


def test_binding_table_is_the_documented_one():
    inv = torch.tensor([1.0, 0.1, 1e-3], dtype=torch.float64)
    t = pkv.rope_table(1000, inv).cpu().numpy()
    ang = np.arange(1000)[:, None] * inv.numpy()
    np.testing.assert_allclose(t, np.concatenate([np.cos(ang), np.sin(ang)], 1), atol=2.0 ** -24)


@pytest.mark.parametrize("kv8", [False, True])
def test_parts_of_one_row_in_place(kv8):
    """q, k and v as slices of one projection's rows, q rotated in place; a layer of a pool of three."""
    c = Case(16, 700, 4, 2, 128, 16, "bf16", kv8, axes=2)
    rows = torch.cat([u16_to_dev(b, "bf16").view(c.N, -1) for b in (c.q, c.k, c.v)], 1)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in rows.split([512, 256, 256], 1))
    b = c.before
    desc = pkv.CacheDesc(b.nb, 16, 2, 128, torch.bfloat16, num_layers=3, kv_int8=kv8)
    one = b.pool.view(np.uint8).reshape(-1)
    pool = torch.from_numpy(np.concatenate([one * 0, one, one * 0])).cuda()
    pkv.rope_reshape_and_cache(q, q, pool, desc, k, v, torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.pos).cuda(),
                               torch.from_numpy(c.cos_sin).cuda(), pair_axis=c.pair_axis, layer=1)
    want = c.expected()
    assert np.array_equal(dev_to_u16(q), want[0])
    assert np.array_equal(dev_to_u16(k), c.k) and np.array_equal(dev_to_u16(v), c.v)
    got = pool.cpu().numpy().reshape(3, -1)
    assert np.array_equal(got[1], want[1].view(np.uint8).reshape(-1)) and not got[0].any() and not got[2].any()


def test_replays_and_another_stream():
    c = Case(17, 90, 4, 2, 128, 16, "f16", axes=3)
    desc = pkv.CacheDesc(c.before.nb, 16, 2, 128, torch.float16)
    t = [u16_to_dev(b, "f16") for b in (c.q, c.k, c.v)]
    pool = torch.from_numpy(c.before.pool.view(np.int16).copy()).cuda()
    args = [torch.from_numpy(x).cuda() for x in (c.slots, c.pos, c.cos_sin)]
    out = torch.zeros_like(t[0])
    call = lambda: pkv.rope_reshape_and_cache(out, t[0], pool, desc, t[1], t[2], *args, pair_axis=c.pair_axis)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    out.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = c.expected()
    assert np.array_equal(dev_to_u16(out), want[0]) and np.array_equal(pool.cpu().numpy().view(np.uint16), want[1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_codes_of_vectors_that_are_not_finite(dtype, pairs):
    """8-bit caches: a NaN element has code 0 beside the codes of the finite ones; a vector with an infinity has codes 0
    and an infinite scale; of NaN alone, codes and scale 0.  What is not rotated agrees with the plain cache writer."""
    c = Case(18, 8, 2, 2, 128, 8, dtype, kv8=True, rot=16, pairs=pairs)
    inf, nan, minf = (0x7F80, 0x7FC0, 0xFF80) if dtype == "bf16" else (0x7C00, 0x7E00, 0xFC00)
    for x in (c.k, c.v):                                             # (dims from 16 on are not rotated)
        x[0, 0, 20], x[1, 1, [40, 127]] = nan, nan
        x[2, 0, 33], x[3, 1, 90], x[4, 0, [21, 60]] = inf, minf, [inf, nan]
        x[5, 1], x[6, 0, :] = nan, minf
        x[0, 1, 77] = nan | 0x8000
    c.k[5, 1], c.k[6, 0] = nan, minf                                 # (and all of a rotated vector)
    f = lambda bits: bits_to_f64(bits, dtype).astype(np.float32)
    n = c.rot // 2
    row = c.cos_sin[c.pos[0]]
    with np.errstate(invalid="ignore"):
        k = step_ref.rotate32(f(c.k), row[:, :n], row[:, n:], c.rot, pairs)
    after = step_ref.Cache(c.before.nb, 8, 2, 128, dtype, True)
    after.pool = c.before.pool.copy()
    for part, x in enumerate((k, f(c.v))):
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            amax = np.fmax.reduce(np.abs(x), -1, keepdims=True)
            amax = np.where(np.isnan(amax), 0, amax).astype(np.float32)
            inv = np.where(amax > 0, np.float32(127) * (np.float32(1) / amax), 0).astype(np.float32)
            y = (x * inv).astype(np.float32)
            codes = np.where(np.isnan(y), 0, np.clip(np.rint(y), -127, 127)).astype(np.int8)
            step_ref.store8(after, codes, (amax * (np.float32(1) / np.float32(127))).astype(np.float32), part, c.slots)
    pool = c.run()[1]
    assert np.array_equal(pool, after.pool)
    # the plain writer's codes and scales of v (its scale is a division, so off by at most a step)
    desc = pkv.CacheDesc(c.before.nb, 8, 2, 128, step_ref.torch_dtype(dtype), kv_int8=True)
    plain = torch.from_numpy(c.before.pool.copy()).cuda()
    pkv.reshape_and_cache(plain, desc, u16_to_dev(c.v, dtype), u16_to_dev(c.v, dtype), torch.from_numpy(c.slots).cuda())
    a, b = after, step_ref.Cache(c.before.nb, 8, 2, 128, dtype, True)
    b.pool = plain.cpu().numpy()
    for i, (block, t) in enumerate(zip(c.slots // 8, c.slots % 8)):
        for h in range(2):
            base = (block * 2 + h) * step_ref.chunk_bytes8(8)
            at = base + step_ref.offsets8(8, [t], 1)[0]
            ca, cb = a.pool[at].view(np.int8).astype(int), b.pool[at].view(np.int8).astype(int)
            assert (np.abs(ca - cb) <= 1).all() and (ca[~np.isfinite(f(c.v)[i, h])] == 0).all() and (cb[~np.isfinite(f(c.v)[i, h])] == 0).all()
        sa, sb = a.scales([block], [t], 1), b.scales([block], [t], 1)
        np.testing.assert_allclose(sa, sb, rtol=2.0 ** -22)


@pytest.mark.parametrize("gap", [0, 8])
def test_output_between_the_rows_it_comes_from(gap):
    """q_out, q, key and value as parts of the same rows, none over another."""
    c = Case(23, 70, 4, 2, 128, 16, "bf16")
    rows = torch.full((c.N, 3 * (512 + gap)), float("nan"), dtype=torch.bfloat16, device="cuda")
    at = lambda i, n: rows[:, i:i + n * 128].unflatten(1, (n, 128))
    q, q_out, k, v = at(0, 4), at(512 + gap, 4), at(2 * (512 + gap), 2), at(2 * (512 + gap) + 256, 2)
    for x, b in ((q, c.q), (k, c.k), (v, c.v)):
        x.copy_(u16_to_dev(b, "bf16"))
    b = c.before
    pool = torch.from_numpy(b.pool.view(np.int16).copy()).cuda()
    pkv.rope_reshape_and_cache(q_out, q, pool, pkv.CacheDesc(b.nb, 16, 2, 128, torch.bfloat16), k, v, torch.from_numpy(c.slots).cuda(),
                               torch.from_numpy(c.pos).cuda(), torch.from_numpy(c.cos_sin).cuda())
    want = c.expected()
    assert np.array_equal(dev_to_u16(q_out), want[0]) and np.array_equal(pool.cpu().numpy().view(np.uint16), want[1])
    for x, bits in ((q, c.q), (k, c.k), (v, c.v)):
        assert np.array_equal(dev_to_u16(x), bits)


def test_single_tokens_of_any_stride():
    """With one token its stride says nothing: heads by tokens, seen as tokens by heads."""
    c = Case(24, 1, 4, 2, 128, 16, "bf16")
    one = lambda bits: u16_to_dev(bits, "bf16").as_strided((1, bits.shape[1], 128), (128, 128, 1))
    b = c.before
    pool = torch.from_numpy(b.pool.view(np.int16).copy()).cuda()
    q = one(c.q)
    pkv.rope_reshape_and_cache(q, q, pool, pkv.CacheDesc(b.nb, 16, 2, 128, torch.bfloat16), one(c.k), one(c.v), torch.from_numpy(c.slots).cuda(),
                               torch.from_numpy(c.pos).cuda(), torch.from_numpy(c.cos_sin).cuda())
    want = c.expected()
    assert np.array_equal(dev_to_u16(q), want[0]) and np.array_equal(pool.cpu().numpy().view(np.uint16), want[1])
