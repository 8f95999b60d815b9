"""pa_extend_scored and pa_decode_scored at the ends of what their interface allows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64
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
