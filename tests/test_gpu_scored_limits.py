"""pa_extend_scored and pa_decode_scored at the ends of what their interface allows."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64, to_bits
from scored_ref import Scored, alibi
from test_gpu_scored import assert_close, decode, desc_of, dev, pool_to_dev, run

pytestmark = pytest.mark.gpu

FAR = 2**31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def values(t):
    return bits_to_f64(dev_to_u16(t), {torch.float16: "f16", torch.bfloat16: "bf16"}[t.dtype])


# ------------------------------------------------------------------ empty spans

@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("kind", ["spans", "cap", "slopes", "both"])
@pytest.mark.parametrize("q_lens,ctx", [([90], [600]), ([3, 20], [700, 400]), ([20] * 90, [400] * 90), ([100] * 50, [500] * 50)])
def test_empty_spans_beside_bad_key_scales(q_lens, ctx, kind, what):
    """8-bit caches: a K scale that is not finite, in a KV tile that every query with a span attends whole.  Queries
    whose span is empty get zero rows all the same: in contexts that are split over SMs and in whole ones, in items of
    one query tile and of two."""
    rng = np.random.default_rng(len(q_lens))
    case = Scored(rng, q_lens, ctx, Hq=6, Hkv=2, D=128, bs=16, dtype="bf16", kv8=True)
    c, n = case.cache, int(case.qsl[-1])
    for s in range(len(ctx)):                                        # position 140 + s % 100, kv head 1
        pos = 140 + s % 100
        at = (int(case.tables[s, pos // 16]) * c.Hkv + 1) * step_ref.chunk_bytes8(16) + 2 * 16 * 128 + 4 * (pos % 16)
        c.pool[at:at + 4] = np.float32(what).reshape(1).view(np.uint8)
    empty = rng.random(n) < 0.4
    first = np.where(empty, FAR, 0).astype(np.int32)
    shape = dict(first=first)
    if kind in ("cap", "both"):
        shape["cap"] = 20.0
    if kind in ("slopes", "both"):
        shape["slopes"] = alibi(6)
    got = values(run(case, 0.1, **shape))
    assert not got[empty].any() and np.isfinite(got[empty]).all()
    with np.errstate(invalid="ignore"):
        out, tol = case.shaped(0.1, **shape)
    assert (np.abs(got[:, :3] - out[:, :3]) <= tol[:, :3]).all()     # the other kv head
    if np.isnan(what):
        assert np.isnan(got[~empty][:, 3:]).all()


# ------------------------------------------------------------------ the ends of the value range under a cap

def saturated(side, cap, spread, dtype="bf16", q_lens=(100, 3), ctx=(300, 200), exponents=(0, 0), share=1.0, seed=0, kv8=False):
    """Chunks whose scores all lie near side * cap * spread (spread 1: at the cap), with values of 2^exponents."""
    rng = np.random.default_rng(seed)
    case = Scored(rng, list(q_lens), list(ctx), Hq=4, Hkv=2, D=128, bs=16, dtype=dtype)
    c = case.cache
    unit = rng.choice([-1.0, 1.0], (1, 128))
    case.q_bits = to_bits(np.broadcast_to(side * unit, (case.T, 4, 128)) * rng.uniform(0.97, 1.0, (case.T, 4, 1)), dtype)
    case.q = bits_to_f64(case.q_bits, dtype)
    for s, n in enumerate(ctx):
        t = np.arange(n)
        for h in range(2):
            base = (case.tables[s, t // 16] * c.Hkv + h) * step_ref.chunk_elements(16, 128)
            c.pool[base[:, None] + step_ref.offsets16(16, 128, t % 16, 0)] = to_bits(unit * rng.uniform(0.97, 1.0, (n, 1)), dtype)
            v = rng.standard_normal((n, 128)) * 2.0 ** rng.uniform(*exponents, (n, 1)) if exponents[0] != exponents[1] else \
                rng.standard_normal((n, 128)) * 2.0 ** exponents[0]
            c.pool[base[:, None] + step_ref.offsets16(16, 128, t % 16, 1)] = to_bits(v, dtype)
    # q.k is 128 up to 6%; scale * 128 / cap = atanh(spread), or 8 (tanh is 1 - 2^-22 there) at the cap
    y = 8.0 if spread >= 1 else math.atanh(spread)
    return case, cap * y / 128


@pytest.mark.parametrize("cap", [5.0, 30.0, 55.0])
@pytest.mark.parametrize("spread", [0.5, 1.0])
@pytest.mark.parametrize("exponent", [-40, -60, -75])
def test_small_values_under_scores_near_the_lower_cap(exponent, spread, cap):
    """Every score of a row is near -cap (or half of it): values far below 1 come back all the same."""
    case, scale = saturated(-1, cap, spread, exponents=(exponent, exponent))
    got = values(run(case, scale, cap=cap))
    out, tol = case.shaped(scale, cap=cap)
    big = np.abs(out).max()
    assert 2.0 ** (exponent - 8) < big < 2.0 ** (exponent + 3)
    # (the bound's floor of 1e-30 is far below these values)
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], out[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("cap", [30.0, 55.0])
@pytest.mark.parametrize("side", [-1, 1])
@pytest.mark.parametrize("exponents", [(40, 40), (100, 100), (-60, 60)])
def test_large_values_under_scores_near_a_cap(exponents, side, cap):
    """Weights of e^cap beside values of 2^100 leave fp32; the results do not."""
    case, scale = saturated(side, cap, 1.0, exponents=exponents)
    assert_close(run(case, scale, cap=cap), case.shaped(scale, cap=cap))


def test_zero_values_under_scores_near_the_lower_cap():
    """Dims that are zero throughout stay zero, whatever the scores."""
    case, scale = saturated(-1, 55.0, 1.0)
    c = case.cache
    for s, n in enumerate((300, 200)):
        t = np.arange(n)
        base = case.tables[s, t // 16] * c.Hkv * step_ref.chunk_elements(16, 128)
        c.pool[base[:, None] + step_ref.offsets16(16, 128, t % 16, 1)[:, 96:]] = 0
    got = run(case, scale, cap=55.0)
    assert_close(got, case.shaped(scale, cap=55.0))
    assert not values(got)[:, :2, 96:].any()


@pytest.mark.parametrize("dtype,kv8", [("f16", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_scores_far_beyond_and_far_below_a_cap(scale, dtype, kv8):
    """Every score is the cap or its opposite; or all of them are nearly 0."""
    rng = np.random.default_rng(4)
    case = Scored(rng, [70, 3], [300, 500], Hq=4, Hkv=2, D=128, bs=16, dtype=dtype, kv8=kv8)
    one = Scored(rng, [1, 1], [300, 500], Hq=4, Hkv=2, D=128, bs=16, dtype=dtype, kv8=kv8)
    for c, got in ((case, run(case, scale, cap=2.0)), (one, decode(one, scale, cap=2.0))):
        got, row = values(got), 0
        for s, n in enumerate(c.q_lens):
            t = np.arange(c.ctx[s])
            k, v = (c.cache.read(c.tables[s, t // 16], t % 16, part) for part in (0, 1))
            for j in range(n):
                m = c.ctx[s] - n + j + 1
                for h in range(4):
                    z = 2.0 * np.sign(k[:m, h // 2] @ c.q[row, h]) if scale > 1 else np.zeros(m)
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    out, size = w @ v[:m, h // 2], w @ np.abs(v[:m, h // 2])
                    # the result's rounding, the weights', and scores off by 2^-20 of 2: 4 2^-20 of every weight; in 16 bits
                    # and fewer the weights' smallest numbers do not matter (they are at least e^-4)
                    u = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
                    tol = u * np.abs(out) + (u + 2.0 ** -16) * size + 2.0 ** -21 * np.abs(v[:m, h // 2]).sum(0)
                    assert (np.abs(got[row, h] - out) <= tol).all()
                row += 1


# ------------------------------------------------------------------ slopes of any size

@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("slopes", [[1e27, -1e27, 1e15, -1e15], [1e8, -1e8, 3e4, -3e4], [3e5, -3e5, 3e6, -2e7]])
def test_steep_slopes(slopes, kv8, cap):
    """A positive slope leaves the nearest attended position, a negative one the farthest, with its value: also where
    slope times distance is far beyond what a power of two can take."""
    rng = np.random.default_rng(1)
    s = np.asarray(slopes, np.float32)
    case = Scored(rng, [260, 3], [900, 5000], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    n = int(case.qsl[-1])
    pos = np.concatenate([np.arange(c - q, c) for q, c in zip(case.q_lens, case.ctx)])
    seq = np.repeat([0, 1], case.q_lens)

    def value(p, h):
        out = np.empty((n, 128))
        for b in (0, 1):
            at = p[seq == b]
            out[seq == b] = case.cache.read(case.tables[b, at // 16], at % 16, 1)[:, h]
        return out

    def expect(got, near, far, rows=slice(None)):
        g = values(got)
        for h in range(4):
            want = value(near if s[h] > 0 else far, h // 2)[rows]
            # one weight of 1; the result's rounding (half of bf16's step of 2^-7); in an 8-bit cache that of the weight,
            # which carries V's scale (half of fp16's step of 2^-10, or of its smallest step 2^-24 beside codes of 127
            # times 2^8 of the tile's largest scale)
            slack = 2.0 ** -8 + (2.0 ** -11 if kv8 else 0)
            assert (np.abs(g[:, h] - want) <= slack * np.abs(want) + (2.0 ** -12 if kv8 else 0)).all(), h

    expect(run(case, 0.1, cap=cap, slopes=s), pos, 0 * pos)
    first = np.maximum(pos - rng.integers(0, 300, n), 0).astype(np.int32)
    expect(run(case, 0.1, cap=cap, slopes=s, first=first), pos, first)
    last = (first + rng.integers(0, 50, n)).astype(np.int32)
    last = np.minimum(last, pos).astype(np.int32)
    expect(run(case, 0.1, cap=cap, slopes=s, first=first, last=last), last, first)
    one = Scored(rng, [1] * 2, [900, 5000], Hq=4, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    case, n, pos, seq = one, 2, np.asarray([899, 4999]), np.asarray([0, 1])
    f = np.asarray([100, 4000], np.int32)
    expect(decode(one, 0.1, cap=cap, slopes=s), pos, 0 * pos)
    expect(decode(one, 0.1, cap=cap, slopes=s, first=f), pos, f)


# ------------------------------------------------------------------ rings and windows of far contexts

def far_ring(rng, kv8, D, Hq, bs=16, ring=12):
    """Contexts longer than their rings, which whole turns more leave as they are; tokens of a turn."""
    case = Scored(rng, [1] * 4, [400, 333, 250, 193], size=2.0, Hq=Hq, Hkv=2, D=D, bs=bs, dtype="bf16", kv8=kv8, ring=ring)
    return case, ring * bs


@pytest.mark.parametrize("D,kv8,Hq", [(128, False, 8), (128, True, 8), (64, False, 8), (128, False, 6)])
@pytest.mark.parametrize("window", [0, 100])
def test_single_tokens_of_far_ring_contexts(window, D, kv8, Hq):
    """A ring holds the newest tokens of contexts near 2^31: the workspace is that of what is attended, and nothing
    behind it is written."""
    rng = np.random.default_rng(2)
    case, turn = far_ring(rng, kv8, D, Hq)
    c, d = case.cache, desc_of(case.cache)
    far = np.int32((2**31 - 1 - 20000) // turn * turn)
    most = int(case.ctx.max()) + int(far)
    span = pkv.decode_window_span(most, 16, window, case.ring)
    need = pkv.decode_scored_workspace_bytes(d, 4, Hq, span)
    assert need < 1 << 26
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    q = u16_to_dev(case.q_bits, "bf16")
    for kw, ref in ((dict(softcap=5.0), dict(cap=5.0)), (dict(slopes=dev(alibi(Hq))), dict(slopes=alibi(Hq)))):
        out, err = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.decode_scored(out, q, pool_to_dev(c), d, dev(case.tables), dev(case.ctx + far), most, 0.1, ws[:need], window=window,
                          ring_blocks=case.ring, dev_err=err, **kw)
        assert pkv.read_device_errors(err) == 0
        assert bool((ws[need:] == 0xA5).all())
        assert_close(out, case.shaped(0.1, window, **ref))


@pytest.mark.parametrize("window,kv8", [(0, False), (100, True)])
def test_windowed_workspaces_are_enough_and_larger_ones_too(window, kv8):
    """A workspace for the span, and one for the whole context as callers had to bring it: the same results."""
    rng = np.random.default_rng(3)
    case = Scored(rng, [1] * 3, [20000, 9000, 700], size=2.0, Hq=8, Hkv=2, D=128, bs=16, dtype="bf16", kv8=kv8)
    d = desc_of(case.cache)
    whole = decode(case, 0.1, window, cap=5.0)
    span = pkv.decode_window_span(20000, 16, window)
    need = pkv.decode_scored_workspace_bytes(d, 3, 8, span)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full_like(whole, 7.0)
    pkv.decode_scored(out, u16_to_dev(case.q_bits, "bf16"), pool_to_dev(case.cache), d, dev(case.tables), dev(case.ctx), 20000, 0.1,
                      ws[:need] if need else None, softcap=5.0, window=window)
    assert_close(out, case.shaped(0.1, window, cap=5.0))
    assert bool((out == whole).all()) and bool((ws[need:] == 0xA5).all())
