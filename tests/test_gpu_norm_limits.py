"""pa_norm_rope_reshape_and_cache at the ends of what its interface allows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import ensure_built, u16_to_dev
from paged_helpers import to_bits
from test_gpu_norm_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pairs,rot", [(False, 128), (True, 32)])
def test_keys_that_are_not_finite_into_an_8_bit_cache(pairs, rot, dtype):
    """They are NaN in the cache, as the norm's results are, and not vectors of zeros that attention would take for keys."""
    nan, inf, minf = {"bf16": (0x7FC0, 0x7F80, 0xFF80), "f16": (0x7E00, 0x7C00, 0xFC00)}[dtype]
    make = lambda: Case(7, 9, 2, 2, 128, 16, dtype, True, rot, pairs=pairs)
    c, d = make(), make()
    d.k[1, 0, 5], d.k[2, 1, 70], d.k[3, 0, 0], d.k[4, 1, 127] = nan, inf, minf, nan
    d.k[5, 0, :] = inf
    d.v[6, 1, 9] = nan                                               # (values are not normed: their codes are as ever)
    bad = np.zeros((9, 2), bool)
    bad[1, 0] = bad[2, 1] = bad[3, 0] = bad[4, 1] = bad[5, 0] = True
    (_, a), (_, b) = c.run(), d.run()
    block, t = c.slots // 16, c.slots % 16
    ka, kb = a.read(block, t, 0), b.read(block, t, 0)
    assert np.array_equal(ka[~bad], kb[~bad])
    assert np.isnan(kb[bad]).any(-1).all()
    va, vb = a.read(block, t, 1), b.read(block, t, 1)
    keep = np.ones((9, 2), bool)
    keep[6, 1] = False
    assert np.array_equal(va[keep], vb[keep])
    # a query that attends such a key gets NaN
    desc = pkv.CacheDesc(b.nb, 16, 2, 128, step_ref.torch_dtype(dtype), kv_int8=True)
    pool = torch.from_numpy(b.pool.copy()).cuda()
    at = int(np.flatnonzero(block == block[2])[0])
    q = u16_to_dev(np.full((1, 2, 128), to_bits(np.ones(1), dtype)[0], np.uint16), dtype)
    out = torch.zeros_like(q)
    tables = torch.tensor([[int(block[at])]], dtype=torch.int32, device="cuda")
    first = torch.tensor([int(t[2])], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([int(t[2]) + 1], dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    pkv.decode_scored(out, q, pool, desc, tables, ctx, 16, 0.1, ws, first_pos=first)
    assert bool(torch.isnan(out[0, 1]).all()) and not bool(torch.isnan(out[0, 0]).any())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("eps", [1.4e-45, 1e-44, 1e-40, 1.2e-38, 1e-32, 1e-24, 1e20, 1e38])
def test_vectors_beside_every_eps(eps, kv8, dtype):
    """Squares that are too small for fp32 beside an eps that is smaller still; and an eps near fp32's end."""
    c = Case(5, 24, 4, 2, 128, 16, dtype, kv8, eps=float(np.float32(eps)))
    rng = np.random.default_rng(8)
    # (sizes whose results are far above bf16's smallest numbers)
    fits = lambda size: size / np.sqrt(max(c.eps, size * size)) > 1e-30
    for name, h in (("q", 4), ("k", 2)):
        x = getattr(c, name)
        for i, size in enumerate((1e-10, 1e-15, 1e-18, 1e-20, 1e-21, 1e-22, 1e-23, 1e-25, 1e-30, 1e-35, 1e15, 1e18, 1e25, 1e38)):
            if dtype == "bf16" and fits(size):
                x[i] = to_bits(rng.uniform(-1, 1, (h, 128)) * size, dtype)
        x[14] = 0
        if dtype == "f16" or fits(9e-41):
            x[15] = 0
            x[15, 0, 77] = 1                                         # the smallest number there is
    if dtype == "bf16":
        c.w = [to_bits(rng.uniform(0.5, 2, 128), dtype) for _ in range(2)]
    c.check()
