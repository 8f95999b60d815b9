"""Single tokens over 8-bit caches whose values are far from 1: weights carry the V scales, and have to keep their bits
whatever those are.  Within the bounds of scored_ref.extend: fp16 weights against the largest product of weight and
scale, two words each, are off by 2^-25 of it at most, which is less than the bound allows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import ensure_built, u16_to_dev
from paged_helpers import bits_to_f64
from scored_ref import Scored, alibi
from test_gpu_scored import assert_close, decode, desc_of, dev, pool_to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def scaled(seed, ctx, factors, G=4, Hkv=2, bs=16, dtype="bf16", size=3.0):
    """Contexts whose V scales are multiplied by 2^factors(n)."""
    rng = np.random.default_rng(seed)
    case = Scored(rng, [1] * len(ctx), ctx, size=size, Hq=G * Hkv, Hkv=Hkv, D=128, bs=bs, dtype=dtype, kv8=True)
    c = case.cache
    f = c.pool.view(np.float32)
    for h in range(Hkv):
        for s, n in enumerate(ctx):
            t = np.arange(n)
            at = ((case.tables[s, t // bs] * c.Hkv + h) * step_ref.chunk_bytes8(bs) + 2 * bs * 128 + step_ref.scale_bytes(bs) + 4 * (t % bs)) // 4
            f[at] = (f[at].astype(np.float64) * 2.0 ** factors(rng, n)).astype(np.float32)
    return case


SIZES = {
    "small": lambda rng, n: np.full(n, -14.0),
    "smaller": lambda rng, n: np.full(n, -30.0),
    "large": lambda rng, n: np.full(n, 25.0),
    "mixed": lambda rng, n: rng.uniform(-14, 0, n),
    "zeros": lambda rng, n: np.where(rng.random(n) < 0.5, -np.inf, -9.0),
    "all zeros": lambda rng, n: np.full(n, -np.inf),
}


def plain(case, scale):
    c, d, S = case.cache, desc_of(case.cache), len(case.ctx)
    q = u16_to_dev(case.q_bits, c.dtype)
    out = torch.full_like(q, float("nan"))
    most = int(case.ctx.max())
    ws = torch.full((max(16, pkv.decode_workspace_bytes(d, S, case.Hq, most)),), 0xff, dtype=torch.uint8, device="cuda")
    pkv.decode_window(out, q, pool_to_dev(c), d, dev(case.tables), dev(case.ctx), most, scale, 0, 0, ws)
    return out


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_shaped_scores(sizes, G):
    case = scaled(1, [3000, 1, 129, 9000], SIZES[sizes], G)
    for shape in (dict(), dict(cap=8.0), dict(slopes=alibi(2 * G)), dict(cap=8.0, slopes=alibi(2 * G))):
        assert_close(decode(case, 0.09, **shape), case.shaped(0.09, **shape), str(list(shape)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_plain_scores(sizes, G, dtype):
    if dtype == "f16" and sizes == "large":
        pytest.skip("values beyond fp16")
    case = scaled(2, [3000, 1, 129, 9000], SIZES[sizes], G, dtype=dtype)
    out, tol = case.shaped(0.09)
    # (results below fp16's normal numbers are off by half of its smallest step)
    assert_close(plain(case, 0.09), (out, tol + (2.0 ** -25 if dtype == "f16" else 0)))


def test_a_token_that_outweighs_all_others_together_with_them():
    """One token of weight 1 and thousands of 2^-12: what those add is as much as what it gives."""
    for kind in ("plain", "shaped"):
        rng = np.random.default_rng(3)
        case = scaled(3, [6000], lambda rng, n: np.full(n, -13.0), G=1, Hkv=1, size=0.0)
        c = case.cache
        # scores: 0 for all tokens but the first, whose key lies along the query
        case.q_bits[:] = 0
        case.q_bits[0, 0, 0] = 0x3F80                                # (1.0 in bf16)
        case.q = bits_to_f64(case.q_bits, "bf16")
        t = np.arange(6000)
        base = case.tables[0, t // 16] * c.Hkv * step_ref.chunk_bytes8(16)
        code0 = base + step_ref.offsets8(16, t % 16, 0)[:, 0]
        c.pool[code0] = 0
        c.pool[code0[0]] = 127
        f = c.pool.view(np.float32)
        f[(base[0] + 2 * 16 * 128) // 4] = np.float32(12 * np.log(2) / 127)
        got = plain(case, 1.0) if kind == "plain" else decode(case, 1.0, cap=1e6)
        assert_close(got, case.shaped(1.0, **({} if kind == "plain" else dict(cap=1e6))), kind)


@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("kind", ["plain", "shaped"])
def test_scales_that_are_not_finite(kind, what):
    """In places that no window reaches they do not matter; a query that attends such a token gets no finite values."""
    window = 300
    for attended in (False, True):
        case = scaled(4, [3000, 700, 129], SIZES["mixed"])
        c = case.cache
        f = c.pool.view(np.float32)
        for s, n in enumerate(case.ctx):
            for part in (0, 1):                                      # of the second kv head: K, V
                pos = n - 100 - part if attended and s == 1 else n - window - 2 - 3 * part
                if pos < 0 or (attended and part == 0 and np.isinf(what)):
                    continue                                         # (an infinite K scale may give weights of 0)
                at = (int(case.tables[s, pos // 16]) * c.Hkv + 1) * step_ref.chunk_bytes8(16) + 2 * 16 * 128 + part * step_ref.scale_bytes(16) + 4 * (pos % 16)
                f[at // 4] = what
        if kind == "shaped":
            got = decode(case, 0.09, window, cap=8.0)
        else:
            d, S = desc_of(c), 3
            q = u16_to_dev(case.q_bits, c.dtype)
            got = torch.full_like(q, 7.0)
            span = pkv.decode_window_span(3000, 16, window)
            ws = torch.full((max(16, pkv.decode_workspace_bytes(d, S, case.Hq, span)),), 0xff, dtype=torch.uint8, device="cuda")
            pkv.decode_window(got, q, pool_to_dev(c), d, dev(case.tables), dev(case.ctx), 3000, 0.09, window, 0, ws)
        with np.errstate(invalid="ignore"):
            out, tol = case.shaped(0.09, window, **(dict(cap=8.0) if kind == "shaped" else {}))
        g = got.double().cpu().numpy()
        bad = np.zeros(out.shape, bool)
        bad[1, 4:] = attended
        assert (np.abs(g - out) <= tol)[~bad].all()
        assert not np.isfinite(g[bad]).any()
