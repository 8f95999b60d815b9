"""pa_extend_scored and pa_decode_scored at the ends of what their interface allows."""
import numpy as np
import pytest
import torch

import step_ref
from gpu_helpers import dev_to_u16, ensure_built
from paged_helpers import bits_to_f64
from scored_ref import Scored, alibi
from test_gpu_scored import run

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
