"""Single tokens of ring contexts at the end of what the decode kernels serve, 2^31 - 16385 tokens, and behind it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
from gpu_helpers import ensure_built, u16_to_dev
from scored_ref import Scored
from test_gpu_scored import assert_close, desc_of, dev, pool_to_dev

pytestmark = pytest.mark.gpu

LONGEST = 2**31 - 16385


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


def calls(case, window, most):
    """decode_window, and decode_scored under a cap, as functions of the contexts."""
    c, d, S = case.cache, desc_of(case.cache), len(case.ctx)
    q, pool, tables = u16_to_dev(case.q_bits, c.dtype), pool_to_dev(c), dev(case.tables)
    span = pkv.decode_window_span(most, c.bs, window, case.ring)
    size = max(pkv.decode_workspace_bytes(d, S, case.Hq, span), pkv.decode_scored_workspace_bytes(d, S, case.Hq, span))
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")

    def plain(ctx, err):
        out = torch.full_like(q, 7.0)
        pkv.decode_window(out, q, pool, d, tables, dev(ctx), most, 0.1, window, case.ring, ws, dev_err=err)
        return out

    def capped(ctx, err):
        out = torch.full_like(q, 7.0)
        pkv.decode_scored(out, q, pool, d, tables, dev(ctx), most, 0.1, ws, softcap=5.0, window=window, ring_blocks=case.ring, dev_err=err)
        return out

    return (plain, {}), (capped, dict(cap=5.0))


@pytest.mark.parametrize("D,kv8,S", [(128, False, 3), (128, True, 3), (64, False, 3), (128, True, 1030)])
@pytest.mark.parametrize("window,ring", [(0, 12), (100, 12), (5000, 400)])
def test_contexts_at_the_end_of_int32(window, ring, D, kv8, S):
    """On tensor cores and on CUDA cores (heads of 64, and 8-bit caches of more than 1024 sequences)."""
    rng = np.random.default_rng(1)
    turn = ring * 16
    # contexts of one turn and a little more, and as far as whole turns go
    ctx = turn + rng.integers(1, 200, S)
    if S > 100 and ring > 100:
        pytest.skip("a pool of 6.5 million tokens")
    case = Scored(rng, [1] * S, ctx, size=2.0, Hq=4, Hkv=2, D=D, bs=16, dtype="f16", kv8=kv8, ring=ring)
    far = ((LONGEST - int(ctx.max())) // turn * turn)
    assert far + 2 * turn > LONGEST - 200
    served = (case.ctx + far).astype(np.int32)
    for call, shape in calls(case, window, 2**31 - 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(served, err)
        assert pkv.read_device_errors(err) == 0
        want = case.shaped(0.1, window, **shape)
        # (8-bit plain scores on CUDA cores: within pa_decode's own tolerance)
        assert_close(got, (want[0], want[1] + (2e-3 if not shape else 0)))
        if D == 64 and shape:
            continue                                                 # a chunk of one token: up to 2^31 - 129
        refused = served.copy()
        refused[1] = 2**31 - 1 if S > 3 else 2**31 - 16384
        got = call(refused, err)
        assert pkv.read_device_errors(err) == pkv.DEVERR_CONTEXT
        assert bool((got[1] == 0).all())
        assert_close(got[[0, 2]], (want[0][[0, 2]], want[1][[0, 2]] + (2e-3 if not shape else 0)))
