"""pa_extend_scored and pa_decode_scored against attention in 64 bits, within bounds derived in scored_ref.extend."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import scored_ref
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64
from scored_ref import Scored, alibi, documents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def pool_to_dev(cache):
    return torch.from_numpy(cache.pool.copy()).cuda() if cache.kv8 else u16_to_dev(cache.pool, cache.dtype)


def desc_of(c):
    return pkv.CacheDesc(c.nb, c.bs, c.Hkv, c.D, step_ref.torch_dtype(c.dtype), kv_int8=c.kv8)


def padded(x, n):
    """Entries for the rows behind the last sequence: read by nobody."""
    return None if x is None else np.concatenate([x, np.full(n - len(x), -77, x.dtype)])


def run(case, scale, window=0, cap=0.0, slopes=None, first=None, last=None, tables=None, ctx=None, qsl=None, max_q=None, err=None, out=None, q=None, ws=None):
    c = case.cache
    q = u16_to_dev(case.q_bits, c.dtype) if q is None else q
    out = torch.full((case.T, case.Hq, c.D), float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    max_q = int(case.q_lens.max()) if max_q is None else max_q
    if ws is None:
        # poisoned: results must not depend on what a workspace held
        ws = torch.full((pkv.extend_scored_workspace_bytes(desc_of(c), len(case.ctx), case.T, case.Hq, max_q),), 0xff, dtype=torch.uint8, device="cuda")
    pkv.extend_scored(out, q, pool_to_dev(c), desc_of(c), dev(case.tables if tables is None else tables), dev(case.ctx if ctx is None else ctx),
                      dev(case.qsl if qsl is None else qsl), max_q, scale, ws, softcap=cap, slopes=dev(slopes), first_pos=dev(padded(first, case.T)),
                      last_pos=dev(padded(last, case.T)), window=window, ring_blocks=case.ring, dev_err=err)
    return out


def decode(case, scale, window=0, cap=0.0, slopes=None, first=None, ctx=None, max_ctx=None, err=None, tables=None):
    c = case.cache
    q = u16_to_dev(case.q_bits, c.dtype)
    S = len(case.ctx)
    max_ctx = max(1, int(case.ctx.max())) if max_ctx is None else max_ctx
    out = torch.full((S, case.Hq, c.D), float("nan"), dtype=q.dtype, device="cuda")
    ws = torch.full((pkv.decode_scored_workspace_bytes(desc_of(c), S, case.Hq, max_ctx),), 0xff, dtype=torch.uint8, device="cuda")
    pkv.decode_scored(out, q, pool_to_dev(c), desc_of(c), dev(case.tables if tables is None else tables), dev(case.ctx if ctx is None else ctx), max_ctx, scale, ws,
                      softcap=cap, slopes=dev(slopes), first_pos=dev(first), window=window, ring_blocks=case.ring, dev_err=err)
    return out


def assert_close(got, want, what=""):
    out, tol = want
    g = bits_to_f64(dev_to_u16(got), {torch.float16: "f16", torch.bfloat16: "bf16"}[got.dtype])[:len(out)]
    bad = ~(np.abs(g - out) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(np.abs(g - out) / tol, nan=np.inf), 0)), out.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bound; worst at {i}: {g[i]!r}, {out[i]!r} +- {tol[i]!r}")


def check(case, scale=None, window=0, **shape):
    scale = 1 / math.sqrt(case.cache.D) if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, scale, window, err=err, **shape)
    assert pkv.read_device_errors(err) == 0
    n = int(case.qsl[-1])
    out, tol = case.shaped(scale, window, **shape)
    assert_close(got[:n], (out[:n], tol[:n]))
    return got


def check_decode(case, scale=None, window=0, **shape):
    scale = 1 / math.sqrt(case.cache.D) if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = decode(case, scale, window, err=err, **shape)
    assert pkv.read_device_errors(err) == 0
    assert_close(got, case.shaped(scale, window, **shape))
    return got


#        q_lens, ctx: single tokens, tile borders, no new tokens, long prefixes
MIX = ([1, 5, 127, 128, 129, 17, 64, 0, 1, 40, 3], [1, 5, 127, 128, 129, 400, 320, 50, 1000, 40, 257])
KINDS = ["cap", "small cap", "slopes", "both", "spans", "all"]


def shape_of(kind, rng, case):
    """cap: scores well inside it; small cap: most of them far outside."""
    shape = {}
    if kind in ("cap", "both", "all"):
        shape["cap"] = 30.0
    if kind == "small cap":
        shape["cap"] = 0.7
    if kind in ("slopes", "both", "all"):
        shape["slopes"] = alibi(case.Hq)
    if kind in ("spans", "all"):
        shape["first"], shape["last"] = documents(rng, case.q_lens, case.ctx, 90, prefix=40, holes=0.1)
    return shape


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 16])
def test_groups(G, D, kv8, dtype, kind):
    rng = np.random.default_rng(900 + G * 10 + D)
    case = Scored(rng, *MIX, size=3.0, Hq=2 * G, Hkv=2, D=D, bs=16, dtype=dtype, kv8=kv8)
    check(case, **shape_of(kind, rng, case))


@pytest.mark.parametrize("bs", [1, 4, 8, 32])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("window,ring", [(0, 0), (50, 0), (1, 0), (200, -1), (40, 2)])
def test_blocks_windows_and_rings(bs, D, kv8, window, ring):
    """ring -1: just long enough for exact windows; 2: so short that early queries find nothing held."""
    rng = np.random.default_rng(bs + window)
    q_lens, ctx = [60, 1, 33, 0, 130], [60, 500, 333, 70, 400]
    if ring < 0:
        ring = -(-(window + 130 - 1) // bs) + 1
    case = Scored(rng, q_lens, ctx, size=3.0, Hq=6, Hkv=2, D=D, bs=bs, dtype="f16", kv8=kv8, ring=ring)
    check(case, window=window, **shape_of("both", rng, case))
    first, last = documents(rng, q_lens, ctx, 200, prefix=90, holes=0.05)
    check(case, window=window, cap=20.0, first=first)
    # (spans that end behind their query, held to the window's start)
    check(case, window=window, slopes=alibi(6), first=first, last=last)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("q_len", [1, 4, 33, 70])
def test_few_rows_over_long_contexts(q_len, kv8, kind):
    """Work split over the context and merged."""
    rng = np.random.default_rng(q_len)
    case = Scored(rng, [q_len, 1, q_len], [4000, 9001, q_len], size=3.0, Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    shape = shape_of(kind, rng, case)
    if "first" in shape:                                             # long documents
        shape["first"], shape["last"] = documents(rng, case.q_lens, case.ctx, 5000, prefix=4500)
    check(case, **shape)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cap", [1e-4, 0.5, 5.0, 50.0, 300.0, 1e6])
def test_caps_of_every_size(cap, dtype, kv8):
    """Scores tens of units apart, below and above the cap; the running maximum rises from tile to tile."""
    rng = np.random.default_rng(3)
    case = Scored(rng, [300, 1], [700, 1500], size=1.0, Hq=4, Hkv=1, D=128, bs=16, dtype=dtype, kv8=kv8)
    check(case, scale=1.0, cap=cap)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale,cap", [(1e-6, 1e-4), (3e-8, 1e-4), (3e-3, 55.0), (3e-3, 56.0), (1e-4, 1e4)])
def test_small_scales_under_caps(scale, cap, dtype, kv8):
    """Quotients of scale and cap whose ninth power leaves fp32, and caps at both sides of those that need no maximum."""
    rng = np.random.default_rng(30)
    case = Scored(rng, [140, 1], [500, 300], size=20.0, Hq=4, Hkv=2, D=128, bs=16, dtype=dtype, kv8=kv8)
    check(case, scale=scale, cap=cap)


@pytest.mark.parametrize("kv8", [False, True])
def test_rows_at_both_sides_of_the_cap(kv8):
    """Query rows of one tile whose scores are tiny, and some hundreds of times the cap."""
    rng = np.random.default_rng(4)
    case = Scored(rng, [200], [600], Hq=2, Hkv=1, D=128, bs=16, dtype="bf16", kv8=kv8)
    case.q_bits = step_ref.to_bits(case.q * np.exp(rng.uniform(-7, 7, (case.T, 2, 1))), "bf16")
    case.q = bits_to_f64(case.q_bits, "bf16")
    check(case, cap=4.0)
    check(case, cap=4.0, slopes=alibi(2))


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("slopes", [[0.0, 0.0, 0.0, 0.0], [3.0, 1e-4, 0.0, 0.3], [-0.01, 0.05, -1e-5, 8.0]])
def test_slopes_of_any_sign(slopes, kv8):
    rng = np.random.default_rng(5)
    s = np.asarray(slopes, np.float32)
    case = Scored(rng, [260, 3], [900, 5000], Hq=4, Hkv=2, D=128, bs=16, dtype="f16", kv8=kv8)
    check(case, slopes=s)
    first, last = documents(rng, case.q_lens, case.ctx, 700, prefix=600)
    check(case, slopes=s, first=first, last=last)


@pytest.mark.parametrize("kv8", [False, True])
def test_far_spans_under_steep_slopes(kv8):
    """Queries that attend only positions far before (and behind) their own: distances count from the nearest one."""
    rng = np.random.default_rng(6)
    case = Scored(rng, [300, 2], [8000, 9000], Hq=4, Hkv=2, D=128, bs=16, dtype="f16", kv8=kv8)
    n = int(case.qsl[-1])
    last = rng.integers(0, 900, n).astype(np.int32)
    check(case, slopes=np.float32([0.5, 0.01, 2.0, 0.1]), last=last)
    check(case, slopes=np.float32([0.5, 0.01, 2.0, 0.1]), first=np.maximum(last - 50, 0), last=last, cap=10.0)


def test_spans_of_any_values():
    """Starts below 0, ends behind the context, empty and inverted spans, extreme numbers; whole calls that attend nothing."""
    rng = np.random.default_rng(7)
    case = Scored(rng, [140, 1, 70], [300, 400, 70], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16")
    n = int(case.qsl[-1])
    lo, hi = -2**31, 2**31 - 1
    check(case, first=np.full(n, lo, np.int32), last=np.full(n, hi, np.int32))
    first, last = rng.integers(-100, 420, n).astype(np.int32), rng.integers(-100, 420, n).astype(np.int32)
    first[rng.integers(0, n, 20)], last[rng.integers(0, n, 20)] = hi, lo
    got = check(case, first=first, last=last)
    ctx = np.repeat(case.ctx, case.q_lens)
    empty = np.maximum(first, 0) > np.minimum(last, ctx - 1)
    assert empty.any() and bool((got[dev(empty)] == 0).all())
    for kw in (dict(first=np.full(n, hi, np.int32)), dict(last=np.full(n, lo, np.int32)), dict(last=np.full(n, -1, np.int32)), dict(first=np.full(n, 420, np.int32))):
        assert bool((check(case, **kw) == 0).all())
    few = case.shaped(0.1, first=first)[0]
    assert np.isfinite(few).all()
    check(case, first=first)
    check(case, last=last)


def test_many_short_sequences():
    rng = np.random.default_rng(8)
    n = 700
    q = rng.integers(0, 4, n)
    case = Scored(rng, q, q + rng.integers(0, 30, n), Hq=2, Hkv=1, D=64, bs=16, dtype="f16")
    for kind in ("cap", "all"):
        check(case, **shape_of(kind, rng, case))


def test_thousands_of_sequences():
    """More sequences than the planner's threads and than its table of first items."""
    rng = np.random.default_rng(50)
    n = 9000
    q = rng.integers(0, 3, n)
    case = Scored(rng, q, q + rng.integers(0, 4, n), Hq=2, Hkv=1, D=64, bs=8, dtype="f16")
    check(case, **shape_of("all", rng, case))
    one = Scored(rng, np.ones(n, int), 1 + rng.integers(0, 4, n), Hq=2, Hkv=1, D=64, bs=8, dtype="f16")
    check_decode(one, cap=2.0)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("bs", [4, 16])
def test_unshaped_calls_are_the_plain_ones(bs, kv8):
    """Without cap, slopes and spans, the bits of pa_extend; spans that say what causality says change nothing either."""
    rng = np.random.default_rng(9)
    case = Scored(rng, *MIX, Hq=8, Hkv=2, D=128, bs=bs, dtype="bf16", kv8=kv8)
    c = case.cache
    plain = torch.full((case.T, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.extend_workspace_bytes(desc_of(c), len(case.ctx), case.T, 8, 129), dtype=torch.uint8, device="cuda")
    pkv.extend(plain, u16_to_dev(case.q_bits, "bf16"), pool_to_dev(c), desc_of(c), dev(case.tables), dev(case.ctx), dev(case.qsl), 129, 0.1, ws)
    assert bool((run(case, 0.1) == plain).all())
    pos = np.concatenate([np.arange(c - q, c) for q, c in zip(case.q_lens, case.ctx)]).astype(np.int32)
    assert_close(run(case, 0.1, first=pos * 0, last=pos), case.shaped(0.1))


def test_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(10)
    case = Scored(rng, [5, 140], [50, 140], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", extra_rows=70)
    got = check(case, **shape_of("all", rng, case))
    assert bool(torch.isnan(got[145:]).all())


def test_strided_queries():
    rng = np.random.default_rng(11)
    case = Scored(rng, [5, 140], [50, 140], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16")
    wide = torch.full((case.T, 4 * 128 + 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = u16_to_dev(case.q_bits, "bf16").view(case.T, -1)
    got = run(case, 0.1, cap=30.0, q=wide[:, :512].unflatten(1, (4, 128)))
    assert_close(got, case.shaped(0.1, cap=30.0))


@pytest.mark.parametrize("kv8", [False, True])
def test_bad_sequences_are_zero_and_the_others_right(kv8):
    rng = np.random.default_rng(12)
    case = Scored(rng, [10, 6, 3, 300, 1], [50, 4, 60, 300, 2000], Hq=4, Hkv=2, D=128, bs=16, dtype="f16", kv8=kv8)
    tables = case.tables.copy()
    tables[2, 3] = case.cache.nb + 7
    tables[4, 90] = -1
    first, last = np.zeros(case.T, np.int32), np.concatenate([np.arange(c - q, c) for q, c in zip(case.q_lens, case.ctx)]).astype(np.int32)
    a = case.qsl
    for shape in (dict(cap=20.0), dict(cap=20.0, slopes=alibi(4), first=first, last=last)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(case, 0.1, tables=tables, err=err, **shape)
        assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK_ID
        for s in (1, 2, 4):
            assert bool((got[a[s]:a[s + 1]] == 0).all()), s
        for s in (0, 3):
            cut = {k: v[a[s]:a[s + 1]] if k in ("first", "last") else v for k, v in shape.items()}
            want = scored_ref.extend(case.q[a[s]:a[s + 1]], case.cache, case.tables[s:s + 1], case.ctx[s:s + 1], [0, a[s + 1] - a[s]], 0.1, **cut)
            assert_close(got[a[s]:a[s + 1]], want, f"sequence {s}")
    # a bad block that no span reaches does not matter
    free = last.copy()
    first[a[2]:a[3]], first[a[4]:a[5]] = 50, 1600
    tables[2, 3], tables[2, 0] = case.tables[2, 3], -5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.1, tables=tables, err=err, first=first, last=free)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    want = scored_ref.extend(case.q[a[2]:a[3]], case.cache, case.tables[2:3], case.ctx[2:3], [0, 3], 0.1, first=first[a[2]:a[3]])
    assert_close(got[a[2]:a[3]], want)


def test_bad_starts_and_long_chunks():
    rng = np.random.default_rng(13)
    case = Scored(rng, [10, 6, 30], [50, 40, 60], Hq=4, Hkv=2, D=128, bs=16, dtype="f16")
    first = np.zeros(case.T, np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.1, max_q=10, err=err, cap=9.0, first=first)    # the third sequence is longer than that
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((got[16:46] == 0).all())
    out, tol = case.shaped(0.1, cap=9.0)
    assert_close(got[:16], (out[:16], tol[:16]))
    for qsl in ([0, 10, 16, 47], [0, 10, 4, 46], [-1, 10, 16, 46], [0, 2**31 - 1, 16, 46]):
        err.zero_()
        run(case, 0.1, qsl=np.asarray(qsl, np.int32), err=err, cap=9.0, first=first, last=first + 3)
        assert pkv.read_device_errors(err) & pkv.DEVERR_CONTEXT


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [4, 16])
@pytest.mark.parametrize("shape", [dict(cap=30.0), dict(slopes=True), dict(spans=True), dict(cap=0.5, slopes=True)])
def test_infinities_and_nan_in_masked_places(shape, bs, dtype):
    """K and V of single tokens hold infinities and NaN: queries that do not attend those tokens are untouched, the others
    get what the formula gives (a capped infinite score is the cap)."""
    rng = np.random.default_rng(bs)
    case = Scored(rng, [90, 3], [600, 50], Hq=6, Hkv=2, D=128, bs=bs, dtype=dtype)
    inf, nan, minf = (0x7F80, 0x7FC0, 0xFF80) if dtype == "bf16" else (0x7C00, 0x7E00, 0xFC00)
    c = case.cache

    def plant(s, pos, part, head, dims, bits):
        block, t = int(case.tables[s, pos // bs]), pos % bs
        base = (block * c.Hkv + head) * step_ref.chunk_elements(bs, c.D)
        c.pool[base + step_ref.offsets16(bs, c.D, [t], part)[0][dims]] = bits

    plant(0, 531, 1, 0, [3, 70], inf)                                # V that the last queries attend
    plant(0, 543, 1, 0, [3], minf)
    plant(0, 545, 0, 1, [5], nan)                                    # K
    plant(0, 20, 1, 0, [9], nan)                                     # V that spans leave out
    kw = {}
    if "cap" in shape:
        kw["cap"] = shape["cap"]
    if "slopes" in shape:
        kw["slopes"] = alibi(6)
    if "spans" in shape:
        kw["first"] = rng.integers(21, 500, 93).astype(np.int32)
        kw["first"][90:] = 0
    with np.errstate(invalid="ignore"):
        out, tol = case.shaped(0.09, **kw)
    got = bits_to_f64(dev_to_u16(run(case, 0.09, **kw)), dtype)
    fine = np.isfinite(out)
    assert fine.sum() < fine.size and fine.mean() > 0.5
    assert (np.abs(got[fine] - out[fine]) <= tol[fine]).all()
    assert (np.isnan(got) == np.isnan(out)).all()
    big = np.isinf(out)
    assert (got[big] == out[big]).all()


@pytest.mark.parametrize("bs", [4, 16])
def test_infinite_keys_under_a_cap(bs):
    """An infinite score is capped: the token has the weight e^cap or e^-cap."""
    rng = np.random.default_rng(14)
    case = Scored(rng, [40], [300], Hq=4, Hkv=2, D=128, bs=bs, dtype="bf16")
    c = case.cache
    at = (int(case.tables[0, 40 // bs]) * c.Hkv) * step_ref.chunk_elements(bs, c.D)
    c.pool[at + step_ref.offsets16(bs, c.D, [40 % bs], 0)[0][5]] = 0x7F80
    with np.errstate(invalid="ignore"):
        out, tol = case.shaped(0.09, cap=3.0)
    got = bits_to_f64(dev_to_u16(run(case, 0.09, cap=3.0)), "bf16")
    # (the bound's sum of |q k| is infinite: 2^-7 of the largest value covers output and weights, 4 2^-16 the rest)
    k = case.cache.read(case.tables[0, np.arange(300) // bs], np.arange(300) % bs, 1)
    assert np.isfinite(out).all() and (np.abs(got - out) <= (2.0 ** -7 + 2.0 ** -14) * np.abs(k).max()).all()


@pytest.mark.parametrize("what", [np.inf, np.nan, 1e6])
@pytest.mark.parametrize("kind", ["cap", "slopes", "spans"])
def test_scales_in_masked_places(kind, what):
    """8-bit caches: single tokens' scales are infinite, NaN or far above all others: queries that do not attend those tokens are
    untouched."""
    rng = np.random.default_rng(15)
    case = Scored(rng, [90, 3], [600, 50], Hq=6, Hkv=2, D=128, bs=16, dtype="bf16", kv8=True)
    c = case.cache

    def plant(pos, part, head):
        block, t = int(case.tables[0, pos // 16]), pos % 16
        at = (block * c.Hkv + head) * step_ref.chunk_bytes8(16) + 2 * 16 * 128 + part * step_ref.scale_bytes(16) + 4 * t
        c.pool[at:at + 4] = np.float32(what).reshape(1).view(np.uint8)

    plant(531, 1, 0)                                                 # V that the last queries attend
    if np.isnan(what):
        plant(545, 0, 1)                                             # K
    kw = shape_of(kind, rng, case)
    if kind == "spans":
        plant(20, 1, 0)
        kw = dict(first=np.concatenate([rng.integers(21, 500, 90), [0, 0, 0]]).astype(np.int32))
    with np.errstate(invalid="ignore"):
        out, tol = case.shaped(0.09, **kw)
    got = bits_to_f64(dev_to_u16(run(case, 0.09, **kw)), "bf16")
    fine = np.isfinite(out)
    assert np.isfinite(what) or 0.2 < fine.mean() < 1
    assert (np.abs(got[fine] - out[fine]) <= tol[fine]).all()
    assert not np.isfinite(got[~np.isfinite(out)]).any()


@pytest.mark.parametrize("kv8", [False, True])
def test_replays_and_streams(kv8):
    """Captured calls with a workspace each, a chunk and single tokens, replayed on two streams at once, and an eager call beside them."""
    rng = np.random.default_rng(16)
    cases = [Scored(rng, [4, 200, 1], [3000, 300, 900], size=3.0, Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8),
             Scored(rng, [1, 1, 1], [3000, 300, 9000], size=3.0, Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)]
    first, last = documents(rng, cases[0].q_lens, cases[0].ctx, 1000, prefix=300)
    shapes = [dict(cap=30.0, slopes=alibi(8), first=first, last=last), dict(cap=30.0, slopes=alibi(8))]
    graphs, outs, streams, keep = [], [], [], []
    for i, (case, shape) in enumerate(zip(cases, shapes)):
        s = torch.cuda.Stream()
        c, d = case.cache, desc_of(case.cache)
        ws = torch.empty(pkv.extend_scored_workspace_bytes(d, 3, case.T, 8, 200), dtype=torch.uint8, device="cuda")
        t = [u16_to_dev(case.q_bits, "bf16"), pool_to_dev(c)] + [dev(x) for x in (case.tables, case.ctx, case.qsl, shape["slopes"], shape.get("first"), shape.get("last"))]
        out = torch.zeros((case.T, 8, 128), dtype=torch.bfloat16, device="cuda")

        def call(i=i, t=t, out=out, ws=ws, d=d):
            if i == 0:
                pkv.extend_scored(out, t[0], t[1], d, t[2], t[3], t[4], 200, 0.1, ws, softcap=30.0, slopes=t[5], first_pos=t[6], last_pos=t[7])
            else:
                pkv.decode_scored(out, t[0], t[1], d, t[2], t[3], 9000, 0.1, ws, softcap=30.0, slopes=t[5])
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
        keep.append((t, ws, call))
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    eager = run(cases[0], 0.1, **shapes[0])
    torch.cuda.synchronize()
    for case, shape, o in zip(cases, shapes, outs):
        assert_close(o, case.shaped(0.1, **shape))
    assert bool((eager == outs[0]).all())                            # results do not depend on timing


@pytest.mark.parametrize("kv8", [False, True])
def test_captured_call_follows_its_lengths_and_spans(kv8):
    """One captured call; lengths, tables, spans, slopes and queries change in place between replays, down to no queries."""
    S, T, max_q = 4, 160, 150
    cases = []
    for seed, (q, ctx) in enumerate([([4, 0, 150, 1], [700, 9, 150, 40]), ([1, 1, 1, 1], [2000, 1, 30, 900]), ([0, 0, 0, 0], [5, 6, 0, 8])]):
        cases.append(Scored(np.random.default_rng(40 + seed), q, ctx, size=2.0, Hq=6, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8, extra_rows=T - sum(q)))
    nb, width = max(c.cache.nb for c in cases), max(c.tables.shape[1] for c in cases)
    desc = pkv.CacheDesc(nb, 16, 2, 128, torch.bfloat16, kv_int8=kv8)
    pool = torch.zeros(pkv.cache_bytes(desc), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    tables, ctx, qsl, err, first, last = i32(S, width), i32(S), i32(S + 1), i32(1), i32(T), i32(T)
    slopes = torch.zeros(6, device="cuda")
    q = torch.zeros(T, 6, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(pkv.extend_scored_workspace_bytes(desc, S, T, 6, max_q), dtype=torch.uint8, device="cuda")
    call = lambda: pkv.extend_scored(out, q, pool, desc, tables, ctx, qsl, max_q, 0.09, ws, softcap=8.0, slopes=slopes, first_pos=first, last_pos=last, dev_err=err)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    rng = np.random.default_rng(44)
    for k in (0, 1, 2, 0):
        c = cases[k]
        f, l = documents(rng, c.q_lens, c.ctx, 400, prefix=100, holes=0.1)
        sl = (rng.random(6) * 0.1).astype(np.float32)
        bits = torch.from_numpy(c.cache.pool.view(np.uint8).copy()).cuda()
        pool.zero_()
        pool[:bits.numel()] = bits
        tables.fill_(-1)
        tables[:, :c.tables.shape[1]] = dev(c.tables)
        for a, b in ((ctx, c.ctx), (qsl, c.qsl), (first, padded(f, T)), (last, padded(l, T)), (slopes, sl)):
            a.copy_(torch.from_numpy(b))
        q.copy_(u16_to_dev(c.q_bits, "bf16"))
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert pkv.read_device_errors(err) == 0
        n = int(c.qsl[-1])
        want, tol = c.shaped(0.09, cap=8.0, slopes=sl, first=f, last=l)
        assert bool((out[n:] == 7).all())
        assert_close(out[:n], (want[:n], tol[:n])) if n else None


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(17)
    case = Scored(rng, [3, 260, 17], [5000, 900, 4100], size=3.0, Hq=8, Hkv=2, D=128, bs=8, dtype="bf16")
    shape = shape_of("all", rng, case)
    first = run(case, 0.09, **shape)
    for _ in range(20):
        assert bool((run(case, 0.09, **shape) == first).all())


def test_long_cache_offsets():
    """Blocks whose byte offset passes 2^32 (a pool of 5 GB)."""
    rng = np.random.default_rng(18)
    case = Scored(rng, [40], [100], Hq=16, Hkv=8, D=128, bs=16, dtype="bf16")
    c = case.cache
    nb = 5 * 2**30 // (8 * 2 * 16 * 128 * 2)
    pool = torch.full((nb * 8 * 2 * 16 * 128,), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool[-c.pool.size:] = u16_to_dev(c.pool, "bf16")
    tables = np.where(case.tables >= 0, case.tables + nb - c.nb, -1).astype(np.int32)
    desc = pkv.CacheDesc(nb, 16, 8, 128, torch.bfloat16)
    q = u16_to_dev(case.q_bits, "bf16")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.extend_scored_workspace_bytes(desc, 1, 40, 16, 40), dtype=torch.uint8, device="cuda")
    pkv.extend_scored(out, q, pool, desc, dev(tables), dev(case.ctx), dev(case.qsl), 40, 0.1, ws, softcap=3.0)
    assert_close(out, case.shaped(0.1, cap=3.0))


def test_positions_near_the_end_of_int32():
    """A ring keeps a window of a context that is billions of tokens long: distances and spans count there too."""
    rng = np.random.default_rng(19)
    ring, bs, window = 12, 16, 100
    case = Scored(rng, [30], [400], Hq=4, Hkv=2, D=128, bs=bs, dtype="f16", ring=ring)
    turn = ring * bs
    far = np.int32((2**31 - 129 - 400) // turn * turn)
    first = np.arange(300, 330).astype(np.int32)
    last = first + 75
    for kw in (dict(slopes=alibi(4)), dict(slopes=alibi(4), first=first, last=last, cap=4.0)):
        moved = {k: v + far if k in ("first", "last") else v for k, v in kw.items()}
        out = run(case, 0.1, window, ctx=case.ctx + far, **moved)
        assert_close(out, case.shaped(0.1, window, **kw))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(case, 0.1, window, ctx=np.asarray([2**31 - 100], np.int32), err=err, cap=4.0)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT and bool((out == 0).all())


@pytest.mark.parametrize("q_lens,prefix,G", [([8192], [0], 4), ([1483], [22277], 8), ([4880], [0], 16), ([12000, 6000], [0, 40000], 16)])
def test_long_chunks_of_one_kv_head(q_lens, prefix, G):
    """One kv head: query tiles are many, some contexts are cut, and every row is written."""
    rng = np.random.default_rng(70 + G)
    ctx = [q + c for q, c in zip(q_lens, prefix)]
    case = Scored(rng, q_lens, ctx, size=3.0, Hq=G, Hkv=1, D=128, bs=16, dtype="bf16")
    first, last = documents(rng, q_lens, ctx, 20000, prefix=5000)
    shape = dict(cap=30.0, first=first, last=last)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(case, 0.09, err=err, **shape)                          # (into NaN)
    assert pkv.read_device_errors(err) == 0
    assert bool(torch.isfinite(got).all())
    for s, q in enumerate(q_lens):
        for j in np.unique(np.concatenate([np.arange(0, 420, 33), rng.integers(0, q, 20), [q - 1]])):
            row = int(case.qsl[s] + j)
            # one token whose own position is j's, over the whole context
            c = int(case.ctx[s])
            lo, hi = scored_ref.spans(c, q, 16, 0, 0, first[case.qsl[s]:], last[case.qsl[s]:])[j]
            want = scored_ref.extend(case.q[row:row + 1], case.cache, case.tables[s:s + 1], [hi + 1], [0, 1], 0.09, cap=30.0, first=[lo], last=[hi])
            assert_close(got[row:row + 1], want, f"sequence {s}, row {j}")


@pytest.mark.parametrize("kv8", [False, True])
def test_tables_that_are_part_of_wider_rows(kv8):
    """A view of the first entries of longer rows: its own width bounds the contexts, not the rows' pitch."""
    rng = np.random.default_rng(90)
    case = Scored(rng, [1, 1, 1], [50, 160, 100], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    W = case.tables.shape[1]
    wide = dev(np.concatenate([case.tables, np.zeros((3, 7), np.int32)], 1))         # (valid ids behind the view)
    c, d = case.cache, desc_of(case.cache)
    q = u16_to_dev(case.q_bits, "bf16")
    ws = torch.empty(pkv.extend_scored_workspace_bytes(d, 3, 3, 4, 1), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fn in (lambda out, ctx: pkv.extend_scored(out, q, pool_to_dev(c), d, wide[:, :W], dev(ctx), dev(case.qsl), 1, 0.1, ws, softcap=5.0, dev_err=err),
               lambda out, ctx: pkv.decode_scored(out, q, pool_to_dev(c), d, wide[:, :W], dev(ctx), 1000, 0.1, ws, softcap=5.0, dev_err=err)):
        out = torch.full_like(q, 7.0)
        fn(out, case.ctx)
        want, tol = case.shaped(0.1, cap=5.0)
        assert_close(out, (want, tol))
        assert pkv.read_device_errors(err) == 0
        ctx = case.ctx.copy()
        ctx[1] = W * 16 + 1
        fn(out, ctx)
        assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
        assert bool((out[1] == 0).all())
        assert_close(out[[0, 2]], (want[[0, 2]], tol[[0, 2]]))


# ------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("kind", ["none"] + KINDS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,kv8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("G", [1, 2, 4, 5, 8, 16])
def test_decode_groups(G, D, kv8, dtype, kind):
    rng = np.random.default_rng(G * 10 + D)
    ctx = [1, 2, 16, 17, 127, 128, 129, 500, 0, 1300]
    case = Scored(rng, [1 if c else 0 for c in ctx], ctx, size=3.0, Hq=2 * G, Hkv=2, D=D, bs=16, dtype=dtype, kv8=kv8, extra_rows=1)
    shape = shape_of(kind, rng, case)
    shape.pop("last", None)
    # the padded sequence has a row too: its query is the one behind the others
    n = len(ctx)
    order = [0, 1, 2, 3, 4, 5, 6, 7, n - 1, 8]
    first = shape.pop("first", None)
    q_bits = case.q_bits
    case.q_bits = q_bits[order]
    f = None if first is None else np.concatenate([first, [0]]).astype(np.int32)[order]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(D)
    got = decode(case, scale, first=f, err=err, **shape)
    assert pkv.read_device_errors(err) == 0
    assert bool((got[8] == 0).all())
    case.q_bits = q_bits
    out, tol = case.shaped(scale, first=first, **shape)
    assert_close(got[[0, 1, 2, 3, 4, 5, 6, 7, 9]], (out[:n - 1], tol[:n - 1]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("G,Hkv", [(1, 4), (4, 1), (8, 2)])
def test_decode_long_contexts(G, Hkv, kv8, kind):
    """Contexts over many SMs, merged; more of them than fit whole."""
    rng = np.random.default_rng(20)
    case = Scored(rng, [1] * 5, [20000, 1, 7000, 12345, 130], size=3.0, Hq=G * Hkv, Hkv=Hkv, D=128, bs=16, dtype="bf16", kv8=kv8)
    shape = shape_of(kind, rng, case)
    shape.pop("last", None)
    if "first" in shape:
        shape["first"] = np.asarray([15000, 0, 6990, 127, 130], np.int32)           # (the last one attends nothing)
    check_decode(case, **shape)


@pytest.mark.parametrize("bs", [1, 2, 8, 32])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("window,ring", [(50, 0), (1, 0), (200, -1), (40, 2)])
def test_decode_windows_and_rings(bs, kv8, window, ring):
    rng = np.random.default_rng(bs + window)
    if ring < 0:
        ring = -(-(window - 1) // bs) + 1
    case = Scored(rng, [1] * 5, [60, 500, 33, 1, 400], size=3.0, Hq=6, Hkv=2, D=128, bs=bs, dtype="f16", kv8=kv8, ring=ring)
    check_decode(case, window=window, cap=10.0, slopes=alibi(6))
    check_decode(case, window=window, cap=0.5, first=np.asarray([30, 480, 33, -4, 390], np.int32))


def test_decode_refused_contexts():
    rng = np.random.default_rng(21)
    case = Scored(rng, [1, 1, 1], [50, 160, 100], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, tol = case.shaped(0.1, cap=5.0)
    got = decode(case, 0.1, cap=5.0, max_ctx=120, err=err)
    assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
    assert bool((got[1] == 0).all())
    assert_close(got[[0, 2]], (want[[0, 2]], tol[[0, 2]]))
    ctx = np.asarray([-7, 160, 0], np.int32)
    got = decode(case, 0.1, cap=5.0, ctx=ctx, err=err)
    assert pkv.read_device_errors(err) == 0
    assert bool((got[[0, 2]] == 0).all())
    assert_close(got[1:2], (want[1:2], tol[1:2]))
    tables = case.tables.copy()
    tables[0, 1] = -1
    got = decode(case, 0.1, cap=5.0, tables=tables, err=err)
    assert pkv.read_device_errors(err) == pkv.DEVERR_BLOCK_ID
    assert bool((got[0] == 0).all())
    assert_close(got[1:], (want[1:], tol[1:]))


@pytest.mark.parametrize("kv8", [False, True])
def test_decode_agrees_with_decode_window(kv8):
    """Without a shape: both within their bounds of the same value."""
    rng = np.random.default_rng(22)
    case = Scored(rng, [1] * 4, [700, 3, 4100, 64], Hq=8, Hkv=2, D=128, bs=16, dtype="f16", kv8=kv8)
    c = case.cache
    scale = 1 / math.sqrt(128)
    got = check_decode(case, window=600)
    q = u16_to_dev(case.q_bits, "f16")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.decode_workspace_bytes(desc_of(c), 4, 8, 4100), dtype=torch.uint8, device="cuda")
    pkv.decode_window(out, q, pool_to_dev(c), desc_of(c), dev(case.tables), dev(case.ctx), 4100, scale, 600, 0, ws)
    _, tol = case.shaped(scale, 600)
    assert bool(((got.double() - out.double()).abs().cpu().numpy() <= 2 * tol + 2e-3).all())


def test_many_short_decodes():
    rng = np.random.default_rng(23)
    n = 1500
    case = Scored(rng, np.ones(n, int), 1 + rng.integers(0, 40, n), Hq=4, Hkv=1, D=128, bs=16, dtype="bf16")
    check_decode(case, cap=20.0, slopes=alibi(4))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("window,bs", [(0, 16), (90, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_layer_over_several_steps(dtype, window, bs, kv8):
    """Lengths -> tables -> normed and rotated q and k into the cache -> shaped attention: prompts with a prefix that sees itself
    whole, a chunk, and single tokens, all on the device.  Attention is checked against 64 bits over the cache as it is."""
    rng = np.random.default_rng(bs + window)
    S, Hq, Hkv, D = 3, 8, 2, 128
    width = 400 // bs
    nb = S * width + 5
    td = step_ref.torch_dtype(dtype)
    desc = pkv.CacheDesc(nb, bs, Hkv, D, td, kv_int8=kv8)
    pool = torch.zeros(pkv.cache_bytes(desc), dtype=torch.uint8, device="cuda")
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")
    tables, free = z(S, width) - 1, torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    nf = z(1) + nb
    lens, err = z(S), z(1)
    table = pkv.rope_table(500, 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D))
    w = [torch.from_numpy(rng.standard_normal(D) * 0.2).to(td).cuda() for _ in range(2)]
    slopes, prefix = alibi(Hq), 40
    for new in ([130, 1, 57], [20, 100, 4], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        new = np.asarray(new, np.int32)
        qsl, slots, pos = z(S + 1), z(T, dt=torch.int64), z(T)
        x = [torch.from_numpy(rng.standard_normal((T, h, D)) * 5).to(td).cuda() for h in (Hq, Hkv, Hkv)]
        pkv.build_tables(qsl, lens, slots, pos, tables, free, nf, nf, desc, lens, dev(new), dev_err=err)
        pkv.norm_rope_reshape_and_cache(x[0], x[0], pool, desc, x[1], x[2], slots, pos, table, w[0], w[1], 1e-6, weight_offset=1.0, dev_err=err)
        out = torch.full_like(x[0], 7.0)
        last = torch.maximum(pos, torch.full_like(pos, prefix - 1))
        if T > S:
            ws = torch.empty(pkv.extend_scored_workspace_bytes(desc, S, T, Hq, int(new.max())), dtype=torch.uint8, device="cuda")
            pkv.extend_scored(out, x[0], pool, desc, tables, lens, qsl, int(new.max()), D ** -0.5, ws, softcap=6.0, slopes=dev(slopes), last_pos=last, window=window,
                              dev_err=err)
        else:
            ws = torch.empty(pkv.decode_scored_workspace_bytes(desc, S, Hq, 400), dtype=torch.uint8, device="cuda")
            pkv.decode_scored(out, x[0], pool, desc, tables, lens, 400, D ** -0.5, ws, softcap=6.0, slopes=dev(slopes), window=window, dev_err=err)
        assert pkv.read_device_errors(err) == 0
        cache = step_ref.Cache(nb, bs, Hkv, D, dtype, kv8)
        cache.pool = pool.cpu().numpy() if kv8 else pool.cpu().numpy().view(np.uint16)
        want = scored_ref.extend(bits_to_f64(dev_to_u16(x[0]), dtype), cache, tables.cpu().numpy(), lens.cpu().numpy(), qsl.cpu().numpy(), D ** -0.5, window, cap=6.0,
                                 slopes=slopes, last=last.cpu().numpy())
        assert_close(out, want)
