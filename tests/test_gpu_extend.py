"""pa_extend against attention in 64 bits, within bounds derived in step_ref.extend."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64
from step_ref import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def pool_to_dev(cache):
    return torch.from_numpy(cache.pool.copy()).cuda() if cache.kv8 else u16_to_dev(cache.pool, cache.dtype)


def run(case, scale, window=0, tables=None, ctx=None, qsl=None, max_q=None, err=None, out=None, q=None, ws=None, pool=None):
    c = case.cache
    desc = pkv.CacheDesc(c.nb, c.bs, c.Hkv, c.D, step_ref.torch_dtype(c.dtype), kv_int8=c.kv8)
    q = u16_to_dev(case.q_bits, c.dtype) if q is None else q
    out = torch.full((case.T, case.Hq, c.D), float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    max_q = int(case.q_lens.max()) if max_q is None else max_q
    if ws is None:
        # poisoned: results must not depend on what a workspace held
        ws = torch.full((pkv.extend_workspace_bytes(desc, len(case.ctx), case.T, case.Hq, max_q),), 0xff, dtype=torch.uint8, device="cuda")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    pkv.extend(out, q, pool_to_dev(c) if pool is None else pool, desc, dev(case.tables if tables is None else tables), dev(case.ctx if ctx is None else ctx),
               dev(case.qsl if qsl is None else qsl), max_q, scale, ws, window=window, ring_blocks=case.ring, dev_err=err)
    return out


def assert_close(got, want, what=""):
    out, tol = want
    g = bits_to_f64(dev_to_u16(got), {torch.float16: "f16", torch.bfloat16: "bf16"}[got.dtype])[:len(out)]
    bad = ~(np.abs(g - out) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(np.abs(g - out) / tol, nan=np.inf), 0)), out.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bound; worst at {i}: {g[i]!r}, {out[i]!r} +- {tol[i]!r}")


def check(case, scale=None, window=0, rows=None, **kw):
    scale = 1 / math.sqrt(case.cache.D) if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, scale, window, err=err, **kw)
    assert pkv.read_device_errors(err) == 0
    n = int(case.qsl[-1])
    out, tol = case.expected(scale, window)
    assert_close(got[:n], (out[:n], tol[:n]))
    return got


#        q_lens, ctx: single tokens, tile borders, no new tokens, long prefixes
MIX = ([1, 5, 127, 128, 129, 17, 64, 0, 1, 40, 3], [1, 5, 127, 128, 129, 400, 320, 50, 1000, 40, 257])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 12, 16])
def test_groups(G, D, kv8, dtype):
    rng = np.random.default_rng(900 + G * 10 + D)
    check(Chunk(rng, *MIX, Hq=2 * G, Hkv=2, D=D, bs=16, dtype=dtype, kv8=kv8))


@pytest.mark.parametrize("bs", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("window,ring", [(0, 0), (50, 0), (1, 0), (200, -1), (40, 2)])
def test_blocks_windows_and_rings(bs, D, kv8, window, ring):
    """ring -1: just long enough for exact windows; 2: so short that early queries find nothing held."""
    rng = np.random.default_rng(bs + window)
    q_lens, ctx = [60, 1, 33, 0, 130], [60, 500, 333, 70, 400]
    if ring < 0:
        ring = -(-(window + 130 - 1) // bs) + 1
    case = Chunk(rng, q_lens, ctx, Hq=6, Hkv=2, D=D, bs=bs, dtype="f16", kv8=kv8, ring=ring)
    check(case, window=window)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_len", [1, 4, 31, 32, 33, 70])
def test_few_rows_over_long_contexts(q_len, dtype, kv8):
    """Work split over the context and merged."""
    rng = np.random.default_rng(q_len)
    check(Chunk(rng, [q_len, 1, q_len], [4000, 9001, q_len], Hq=8, Hkv=2, D=128, bs=16, dtype=dtype, kv8=kv8))


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_scores(dtype, kv8):
    """Scores tens of units apart: the running maximum rises from tile to tile."""
    rng = np.random.default_rng(3)
    check(Chunk(rng, [300, 1], [700, 1500], Hq=4, Hkv=1, D=128, bs=16, dtype=dtype, kv8=kv8), scale=1.0)


def test_tiny_scale_and_constant_keys():
    rng = np.random.default_rng(4)
    check(Chunk(rng, [9, 200], [400, 200], Hq=4, Hkv=2, D=64, bs=8, dtype="bf16"), scale=1e-6)
    check(Chunk(rng, [9, 200], [400, 200], Hq=4, Hkv=2, D=128, bs=8, dtype="f16", scale_k=0.0))
    check(Chunk(rng, [9, 200], [400, 200], Hq=4, Hkv=2, D=128, bs=8, dtype="f16", kv8=True, scale_k=0.0))


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    n = 700
    q = rng.integers(0, 4, n)
    check(Chunk(rng, q, q + rng.integers(0, 30, n), Hq=2, Hkv=1, D=64, bs=16, dtype="f16"))


def test_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(6)
    case = Chunk(rng, [5, 140], [50, 140], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", extra_rows=70)
    got = check(case)
    assert bool(torch.isnan(got[145:]).all())


def test_strided_queries():
    rng = np.random.default_rng(7)
    case = Chunk(rng, [5, 140], [50, 140], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16")
    wide = torch.full((case.T, 4 * 128 + 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = u16_to_dev(case.q_bits, "bf16").view(case.T, -1)
    check(case, q=wide[:, :512].unflatten(1, (4, 128)))


@pytest.mark.parametrize("D", [64, 128])
def test_outputs_aligned_to_16_bytes_alone(D):
    rng = np.random.default_rng(9)
    case = Chunk(rng, [5, 140, 1], [50, 140, 9000], Hq=4, Hkv=2, D=D, bs=16, dtype="bf16")
    n = case.T * 4 * D
    room = torch.full((n + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert room.data_ptr() % 32 == 0
    check(case, out=room[8:8 + n].view(case.T, 4, D))
    assert bool(torch.isnan(room[:8]).all()) and bool(torch.isnan(room[8 + n:]).all())


@pytest.mark.parametrize("kv8", [False, True])
def test_bad_sequences_are_zero_and_the_others_right(kv8):
    rng = np.random.default_rng(8)
    case = Chunk(rng, [10, 6, 3, 300, 1], [50, 4, 60, 300, 2000], Hq=4, Hkv=2, D=128, bs=16, dtype="f16", kv8=kv8)
    ctx, tables = case.ctx.copy(), case.tables.copy()
    tables[2, 3] = case.cache.nb + 7
    tables[4, 90] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.1, tables=tables, ctx=ctx, err=err)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK_ID
    a = case.qsl
    case.ctx[1] = 6                                                  # (the reference cannot state q_len > ctx)
    tables[1, 0] = 0
    case.q_lens[[1, 2, 4]] = 0
    for s in (1, 2, 4):
        assert bool((got[a[s]:a[s + 1]] == 0).all()), s
    for s in (0, 3):
        sub = step_ref.extend(case.q[a[s]:a[s + 1]], case.cache, case.tables[s:s + 1], case.ctx[s:s + 1], [0, a[s + 1] - a[s]], 0.1)
        assert_close(got[a[s]:a[s + 1]], sub, f"sequence {s}")


def test_bad_starts_and_long_chunks():
    rng = np.random.default_rng(9)
    case = Chunk(rng, [10, 6, 30], [50, 40, 60], Hq=4, Hkv=2, D=128, bs=16, dtype="f16")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.1, max_q=10, err=err)                          # the third sequence is longer than that
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((got[16:46] == 0).all())
    out, tol = case.expected(0.1)
    assert_close(got[:16], (out[:16], tol[:16]))
    for qsl in ([0, 10, 16, 47], [0, 10, 4, 46], [-1, 10, 16, 46], [0, 2**31 - 1, 16, 46]):
        err.zero_()
        out_t = torch.full((case.T, 4, 128), 7.0, dtype=torch.float16, device="cuda")
        run(case, 0.1, qsl=np.asarray(qsl, np.int32), err=err, out=out_t)
        assert pkv.read_device_errors(err) & pkv.DEVERR_CONTEXT
    ctx = case.ctx.copy()
    ctx[0] = case.tables.shape[1] * 16 + 1                           # past its row
    err.zero_()
    got = run(case, 0.1, ctx=ctx, err=err)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((got[:10] == 0).all())


@pytest.mark.parametrize("kv8", [False, True])
def test_replays_and_streams(kv8):
    """Two captured calls with a workspace each, replayed on two streams at once, and an eager call beside them."""
    rng = np.random.default_rng(10)
    cases = [Chunk(rng, [4, 200, 1], [3000, 300, 900], Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8) for _ in range(2)]
    graphs, outs, streams, keep = [], [], [], []
    for case in cases:
        s = torch.cuda.Stream()
        c = case.cache
        desc = pkv.CacheDesc(c.nb, c.bs, c.Hkv, c.D, torch.bfloat16, kv_int8=c.kv8)
        ws = torch.empty(pkv.extend_workspace_bytes(desc, 3, case.T, 8, 200), dtype=torch.uint8, device="cuda")
        t = [u16_to_dev(case.q_bits, "bf16"), pool_to_dev(c)] + [torch.from_numpy(x).cuda() for x in (case.tables, case.ctx, case.qsl)]
        out = torch.zeros((case.T, 8, 128), dtype=torch.bfloat16, device="cuda")
        call = lambda: pkv.extend(out, t[0], t[1], desc, t[2], t[3], t[4], 200, 0.1, ws)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call()
        graphs.append(g)
        outs.append(out)
        streams.append(s)
        keep.append((t, ws))
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    eager = run(cases[0], 0.1)
    torch.cuda.synchronize()
    for case, o in zip(cases, outs):
        assert_close(o, case.expected(0.1))
    assert bool((eager == outs[0]).all())                            # results do not depend on timing


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(11)
    case = Chunk(rng, [3, 260, 17], [5000, 900, 4100], Hq=8, Hkv=2, D=128, bs=8, dtype="bf16")
    first = run(case, 0.09)
    for _ in range(20):
        assert bool((run(case, 0.09) == first).all())


def test_long_cache_offsets():
    """Blocks whose byte offset passes 2^32 (a pool of 5 GB)."""
    rng = np.random.default_rng(12)
    case = Chunk(rng, [40], [100], Hq=16, Hkv=8, D=128, bs=16, dtype="bf16")
    c = case.cache
    nb = 5 * 2**30 // (8 * 2 * 16 * 128 * 2)
    pool = torch.full((nb * 8 * 2 * 16 * 128,), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = c.pool.size
    pool[-n:] = u16_to_dev(c.pool, "bf16")
    tables = np.where(case.tables >= 0, case.tables + nb - c.nb, -1).astype(np.int32)
    desc = pkv.CacheDesc(nb, 16, 8, 128, torch.bfloat16)
    q = u16_to_dev(case.q_bits, "bf16")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.extend_workspace_bytes(desc, 1, 40, 16, 40), dtype=torch.uint8, device="cuda")
    pkv.extend(out, q, pool, desc, *[torch.from_numpy(x).cuda() for x in (tables, case.ctx, case.qsl)], 40, 0.1, ws)
    assert_close(out, case.expected(0.1))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_agrees_with_prefill(dtype):
    """The same chunk through pa_prefill: both within their bounds of the same value."""
    rng = np.random.default_rng(13)
    case = Chunk(rng, [100, 300], [400, 300], Hq=8, Hkv=2, D=128, bs=16, dtype=dtype)
    c = case.cache
    got = check(case)
    desc = pkv.CacheDesc(c.nb, 16, 2, 128, step_ref.torch_dtype(dtype))
    q = u16_to_dev(case.q_bits, dtype)
    out = torch.empty_like(q)
    pkv.prefill(out, q, pool_to_dev(c), desc, *[torch.from_numpy(x).cuda() for x in (case.tables, case.ctx, case.qsl)], 300, 1 / math.sqrt(128))
    _, tol = case.expected(1 / math.sqrt(128))
    assert bool(((got.double() - out.double()).abs().cpu().numpy() <= 2 * tol).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [4, 16])
@pytest.mark.parametrize("q_lens,ctx,window", [([40, 3], [300, 50], 0), ([90, 1], [4000, 20], 0), ([40, 200], [900, 1200], 100)])
def test_infinities_and_nan_in_masked_places(q_lens, ctx, window, bs, dtype):
    """K and V of single tokens hold infinities and NaN: queries that do not attend those tokens are untouched,
    the others get what the formula gives."""
    rng = np.random.default_rng(bs + window)
    case = Chunk(rng, q_lens, ctx, Hq=6, Hkv=2, D=128, bs=bs, dtype=dtype)
    inf, nan, minf = (0x7F80, 0x7FC0, 0xFF80) if dtype == "bf16" else (0x7C00, 0x7E00, 0xFC00)
    c = case.cache

    def plant(s, pos, part, head, dims, bits):
        block, t = int(case.tables[s, pos // bs]), pos % bs
        base = (block * c.Hkv + head) * step_ref.chunk_elements(bs, c.D)
        c.pool[base + step_ref.offsets16(bs, c.D, [t], part)[0][dims]] = bits

    first = ctx[0] - q_lens[0]
    plant(0, first + 21, 1, 0, [3, 70], inf)                         # V that the last queries attend
    plant(0, first + 33, 1, 0, [3], minf)
    plant(0, first + 35, 0, 1, [5], nan)                             # K
    if window:
        plant(0, first - window + 10, 1, 1, [9], nan)                # leaves the window of the later queries
        plant(0, first - window - 1, 1, 0, [1], nan)                 # attended by nobody
    out, tol = case.expected(0.09, window)
    got = bits_to_f64(dev_to_u16(run(case, 0.09, window)), dtype)
    fine = np.isfinite(out)
    assert fine.sum() < fine.size and fine.mean() > 0.5
    assert (np.abs(got[fine] - out[fine]) <= tol[fine]).all()
    assert (np.isnan(got) == np.isnan(out)).all()
    big = np.isinf(out)
    assert (got[big] == out[big]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [1, 16])
@pytest.mark.parametrize("what", [np.inf, np.nan, 1e6])
@pytest.mark.parametrize("q_lens,ctx,window", [([40, 3], [300, 50], 0), ([90, 1], [4000, 20], 0), ([40, 200], [900, 1200], 100)])
def test_scales_in_masked_places(q_lens, ctx, window, what, bs, dtype):
    """8-bit caches: single tokens' scales are infinite, NaN or far above all others: queries that do not attend
    those tokens are untouched."""
    rng = np.random.default_rng(60 + bs + window)
    case = Chunk(rng, q_lens, ctx, Hq=6, Hkv=2, D=128, bs=bs, dtype=dtype, kv8=True)
    c = case.cache

    def plant(s, pos, part, head):
        block, t = int(case.tables[s, pos // bs]), pos % bs
        at = (block * c.Hkv + head) * step_ref.chunk_bytes8(bs) + 2 * bs * 128 + part * step_ref.scale_bytes(bs) + 4 * t
        c.pool[at:at + 4] = np.float32(what).reshape(1).view(np.uint8)

    first = ctx[0] - q_lens[0]
    plant(0, first + 21, 1, 0)                                       # V that the last queries attend
    if np.isnan(what):
        plant(0, first + 35, 0, 1)                                   # K
    if window:
        plant(0, first - window + 10, 1, 1)                          # leaves the window of the later queries
        plant(0, first - window - 1, 1, 0)                           # attended by nobody
    with np.errstate(invalid="ignore"):
        out, tol = case.expected(0.09, window)
    got = bits_to_f64(dev_to_u16(run(case, 0.09, window)), dtype)
    fine = np.isfinite(out) & (np.abs(out) <= np.finfo(np.float16).max if dtype == "f16" else True)
    assert np.isfinite(what) or 0.2 < fine.mean() < 1
    assert (np.abs(got[fine] - out[fine]) <= tol[fine]).all()
    assert not np.isfinite(got[~np.isfinite(out)]).any()


@pytest.mark.parametrize("kv8", [False, True])
def test_captured_call_follows_its_lengths(kv8):
    """One captured call; lengths, tables and queries change in place between replays, down to no queries at all."""
    S, T, max_q = 5, 200, 150
    cases = []
    for seed, (q, ctx) in enumerate([([4, 0, 150, 1, 3], [700, 9, 150, 40, 3]), ([1, 1, 1, 1, 1], [2000, 1, 30, 900, 17]),
                                     ([0, 0, 0, 0, 0], [5, 6, 0, 8, 9]), ([0, 130, 0, 2, 60], [0, 200, 0, 3000, 60])]):
        cases.append(Chunk(np.random.default_rng(40 + seed), q, ctx, Hq=6, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8,
                           extra_rows=T - sum(q)))
    nb, width = max(c.cache.nb for c in cases), max(c.tables.shape[1] for c in cases)
    desc = pkv.CacheDesc(nb, 16, 2, 128, torch.bfloat16, kv_int8=kv8)
    pool = torch.zeros(pkv.cache_bytes(desc), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    tables, ctx, qsl, err = i32(S, width), i32(S), i32(S + 1), i32(1)
    q = torch.zeros(T, 6, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(pkv.extend_workspace_bytes(desc, S, T, 6, max_q), dtype=torch.uint8, device="cuda")
    call = lambda: pkv.extend(out, q, pool, desc, tables, ctx, qsl, max_q, 0.09, ws, dev_err=err)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    for k in (0, 1, 2, 3, 0):
        c = cases[k]
        bits = torch.from_numpy(c.cache.pool.view(np.uint8).copy()).cuda()
        pool.zero_()
        pool[:bits.numel()] = bits
        tables.fill_(-1)
        tables[:, :c.tables.shape[1]] = torch.from_numpy(c.tables).cuda()
        ctx.copy_(torch.from_numpy(c.ctx))
        qsl.copy_(torch.from_numpy(c.qsl))
        q.copy_(u16_to_dev(c.q_bits, "bf16"))
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert pkv.read_device_errors(err) == 0
        n = int(c.qsl[-1])
        want, tol = c.expected(0.09)
        assert bool((out[n:] == 7).all())
        assert_close(out[:n], (want[:n], tol[:n])) if n else None


def test_thousands_of_sequences():
    """More sequences than the planner's threads and than its table of first items."""
    rng = np.random.default_rng(50)
    n = 9000
    q = rng.integers(0, 3, n)
    check(Chunk(rng, q, q + rng.integers(0, 4, n), Hq=2, Hkv=1, D=64, bs=8, dtype="f16"))


@pytest.mark.parametrize("kv8", [False, True])
def test_layers_of_one_pool(kv8):
    rng = np.random.default_rng(51)
    case = Chunk(rng, [20, 140], [90, 300], Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    c = case.cache
    one = pkv.cache_bytes(pkv.CacheDesc(c.nb, 16, 2, 128, torch.bfloat16, kv_int8=kv8))
    desc = pkv.CacheDesc(c.nb, 16, 2, 128, torch.bfloat16, num_layers=3, layer_stride_bytes=one + 48, kv_int8=kv8)
    pool = torch.zeros(2 * (one + 48) + one, dtype=torch.uint8, device="cuda")
    pool[2 * (one + 48):] = torch.from_numpy(c.pool.view(np.uint8).reshape(-1).copy()).cuda()
    q = u16_to_dev(case.q_bits, "bf16")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.extend_workspace_bytes(desc, 2, case.T, 8, 140), dtype=torch.uint8, device="cuda")
    pkv.extend(out, q, pool, desc, *[torch.from_numpy(x).cuda() for x in (case.tables, case.ctx, case.qsl)], 140, 0.1, ws, layer=2)
    assert_close(out, case.expected(0.1))


def test_positions_near_the_end_of_int32():
    """A ring keeps a window of a context that is billions of tokens long; contexts past 2^31 - 129 are refused."""
    rng = np.random.default_rng(52)
    ring, bs, window = 12, 16, 100
    case = Chunk(rng, [30], [400], Hq=4, Hkv=2, D=128, bs=bs, dtype="f16", ring=ring)
    # the same pool read as a context 2^31 - 512 + ... tokens long: a shift by whole turns of the ring
    turn = ring * bs
    far = (2**31 - 129 - 400) // turn * turn
    out = run(case, 0.1, window, ctx=case.ctx + np.int32(far))
    assert_close(out, case.expected(0.1, window))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(case, 0.1, window, ctx=np.asarray([2**31 - 100], np.int32), err=err)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT and bool((out == 0).all())


def test_very_small_and_large_value_scales():
    """8-bit caches whose V scales span many powers of two, zero vectors among them."""
    rng = np.random.default_rng(53)
    case = Chunk(rng, [40, 3], [700, 300], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", kv8=True)
    c = case.cache
    scales = c.pool.view(np.float32)
    for block in range(c.nb):
        for h in range(c.Hkv):
            at = ((block * c.Hkv + h) * step_ref.chunk_bytes8(16) + 2 * 16 * 128 + step_ref.scale_bytes(16)) // 4
            scales[at:at + 16] *= np.float32(2.0) ** rng.integers(-40, 12, 16).astype(np.float32)
            if block % 5 == 0:
                scales[at:at + 16] = 0
    check(case)


@pytest.mark.parametrize("q_lens,prefix,G", [([8192], [0], 4), ([1483], [22277], 8), ([4880], [0], 16), ([7057], [0], 8),
                                             ([12000, 6000], [0, 40000], 16), ([21000], [0], 1)])
def test_long_chunks_of_one_kv_head(q_lens, prefix, G):
    """One kv head: query tiles are many, some contexts are cut, and every row is written."""
    rng = np.random.default_rng(70 + G)
    ctx = [q + c for q, c in zip(q_lens, prefix)]
    case = Chunk(rng, q_lens, ctx, Hq=G, Hkv=1, D=128, bs=16, dtype="bf16")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.09, err=err)                                   # (into NaN)
    assert pkv.read_device_errors(err) == 0
    assert bool(torch.isfinite(got).all())
    for s, q in enumerate(q_lens):
        for j in np.unique(np.concatenate([np.arange(0, 420, 13), rng.integers(0, q, 30), [q - 1]])):
            row = int(case.qsl[s] + j)
            want = step_ref.extend(case.q[row:row + 1], case.cache, case.tables[s:s + 1], [prefix[s] + j + 1], [0, 1], 0.09)
            assert_close(got[row:row + 1], want, f"sequence {s}, row {j}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [4, 16])
@pytest.mark.parametrize("q_len,ctx", [(40, 300), (90, 4000)])
def test_infinite_keys(q_len, ctx, bs, dtype):
    """The first attended key holds an infinity: its score is -inf for queries of one sign, whose rows are the
    attention over the other positions, and +inf for the others, whose rows the formula leaves undefined."""
    rng = np.random.default_rng(80 + bs)
    case = Chunk(rng, [q_len, 3], [ctx, 50], Hq=4, Hkv=2, D=128, bs=bs, dtype=dtype)
    c = case.cache
    at = int(case.tables[0, 0]) * c.Hkv * step_ref.chunk_elements(bs, c.D)          # position 0, kv head 0
    c.pool[at + step_ref.offsets16(bs, c.D, [0], 0)[0][5]] = 0x7F80 if dtype == "bf16" else 0x7C00
    got = run(case, 0.09)
    for j in range(q_len):
        pos = ctx - q_len + j
        # a window of pos tokens leaves position 0 out
        out, tol = step_ref.extend(case.q[j:j + 1], c, case.tables[:1], [pos + 1], [0, 1], 0.09, window=pos)
        low = case.q[j, :2, 5] < 0
        low = np.concatenate([low, [True, True]])                                   # (kv head 1 is as it was)
        g = bits_to_f64(dev_to_u16(got[j]), dtype)
        assert (np.abs(g - out[0])[:2][low[:2]] <= tol[0][:2][low[:2]]).all(), j
        assert np.isnan(g[:2][~low[:2]]).all(), j
    tail = [case.q_lens[0], case.q_lens[0] + 3]
    assert_close(got[tail[0]:tail[1]], step_ref.extend(case.q[tail[0]:tail[1]], c, case.tables[1:], [50], [0, 3], 0.09))


@pytest.mark.parametrize("kv8", [False, True])
def test_tables_that_are_part_of_wider_rows(kv8):
    """A view of the first entries of longer rows: its own width bounds the contexts, not the rows' pitch."""
    rng = np.random.default_rng(90)
    case = Chunk(rng, [10, 40, 3], [50, 160, 100], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    W = case.tables.shape[1]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    wide = dev(np.concatenate([case.tables, np.zeros((3, 7), np.int32)], 1))         # (valid ids behind the view)
    c = case.cache
    desc = pkv.CacheDesc(c.nb, 16, 2, 128, torch.bfloat16, kv_int8=kv8)
    q = u16_to_dev(case.q_bits, "bf16")
    ws = torch.empty(pkv.extend_workspace_bytes(desc, 3, case.T, 4, 40), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(ctx, **kw):
        out = torch.full_like(q, 7.0)
        pkv.extend(out, q, pool_to_dev(c), desc, wide[:, :W], dev(ctx), dev(case.qsl), 40, 0.1, ws, dev_err=err, **kw)
        return out
    assert_close(call(case.ctx), case.expected(0.1))
    assert pkv.read_device_errors(err) == 0
    ctx = case.ctx.copy()
    ctx[1] = W * 16 + 1
    got = call(ctx)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((got[10:50] == 0).all())
    want, tol = case.expected(0.1)
    assert_close(got[:10], (want[:10], tol[:10]))
    assert_close(got[50:], (want[50:], tol[50:]))
    with pytest.raises(pkv.PagedKVError):
        call(case.ctx, ring_blocks=W + 1)


def test_single_tokens_of_any_stride():
    """With one token its stride says nothing: heads by tokens, seen as tokens by heads."""
    rng = np.random.default_rng(91)
    case = Chunk(rng, [1], [50], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16")
    q = u16_to_dev(case.q_bits, "bf16").transpose(0, 1).contiguous().transpose(0, 1)
    q = q.as_strided((1, 4, 128), (128, 128, 1))
    check(case, q=q)


@pytest.mark.parametrize("small", [2.0 ** -16, 2.0 ** -21])
@pytest.mark.parametrize("q_len,ctx", [(1, 200), (40, 300), (3, 5000)])
def test_attended_tokens_with_small_value_scales(q_len, ctx, small):
    """8-bit caches: nearly all weight falls on a token whose V is far smaller than its neighbours'.  The row is that
    V: off by the output's rounding (2^-8), and its weight's -- stored at 2^7 times the ratio of the scales, which is at
    least 2^-22 here: 2^-25 / 2^-15."""
    rng = np.random.default_rng(92)
    case = Chunk(rng, [q_len], [ctx], Hq=2, Hkv=1, D=128, bs=16, dtype="bf16", kv8=True)
    c, at = case.cache, 130
    case.q_bits[:] = case.q_bits[:1, :1]                             # one query direction
    case.q = bits_to_f64(case.q_bits, "bf16")
    slot = np.asarray([int(case.tables[0, at // 16]) * 16 + at % 16], np.int64)
    v = np.sign(rng.standard_normal((1, 1, 128))) * rng.uniform(0.5, 4, (1, 1, 128)) * small
    assert c.write(case.q_bits[:1, :1], step_ref.to_bits(v, "bf16"), slot) == 0
    got = bits_to_f64(dev_to_u16(run(case, 1.0)), "bf16")            # scores 128 +- 23 and 0 +- 12
    want = c.read(slot // 16, slot % 16, 1)[0, 0]
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -16) * np.abs(want)).all()
