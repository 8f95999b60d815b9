"""The operators of normed heads and shaped scores without a GPU: their references against independent statements,
and the refusals of their entry points.  No call here reaches a kernel launch."""
import ctypes

import numpy as np
import pytest
import torch

import scored_ref
import step_ref
from paged_kv_cache_168_gb300 import _lib, build as build_mod
from paged_kv_cache_168_gb300._lib import CacheDesc

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def V(x=FAKE):
    return ctypes.c_void_p(x)


def _desc(**kw):
    base = dict(num_blocks=16, block_size=16, num_kv_heads=2, head_size=128, dtype=torch.float16)
    base.update(kw)
    return ctypes.byref(CacheDesc(**base).c())


# ------------------------------------------------------------------ references

def test_norm_reference():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 3, 64)), rng.standard_normal(64)
    y = scored_ref.normed(x, None, 0, 0.0)
    np.testing.assert_allclose((y * y).sum(-1), 64, rtol=1e-12)               # of length sqrt(D) ...
    np.testing.assert_allclose(y, scored_ref.normed(x * 1e9, None, 0, 0.0), rtol=1e-12)
    np.testing.assert_allclose(y[0, 0] * x[0, 0, 0], x[0, 0] * y[0, 0, 0], rtol=1e-9)   # ... and x's direction
    np.testing.assert_allclose(scored_ref.normed(x, w, 1, 1e-6), scored_ref.normed(x, w + 1, 0, 1e-6))
    np.testing.assert_allclose(scored_ref.normed(x * 0, w, 1, 1e-6), 0)


def test_unshaped_reference_is_the_plain_chunk():
    rng = np.random.default_rng(1)
    case = scored_ref.Scored(rng, [5, 0, 9], [40, 3, 9], Hq=4, Hkv=2, D=64, bs=8, dtype="f16")
    for window in (0, 7):
        a, b = case.shaped(0.1, window)[0], case.expected(0.1, window)[0]
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-14)


def test_shaped_reference():
    rng = np.random.default_rng(2)
    case = scored_ref.Scored(rng, [12], [30], Hq=2, Hkv=1, D=64, bs=8, dtype="f16", size=8.0)
    # a far cap changes nothing, a near one bounds the scores: weights within a factor e^(2c) of each other
    np.testing.assert_allclose(case.shaped(0.1, cap=1e6)[0], case.expected(0.1)[0], rtol=1e-4, atol=1e-6)
    flat = case.shaped(0.1, cap=1e-3)[0]
    k = case.cache.read(case.tables[0, np.arange(30) // 8], np.arange(30) % 8, 1)[:, 0]
    for j in range(12):
        np.testing.assert_allclose(flat[j, 0], k[:19 + j].mean(0), atol=5e-3)
    # a steep slope leaves the query's own token; a negative one the first
    steep = case.shaped(0.01, slopes=[100.0, -100.0])[0]
    for j in range(12):
        np.testing.assert_allclose(steep[j, 0], k[18 + j], atol=1e-9)
        np.testing.assert_allclose(steep[j, 1], k[0], atol=1e-9)
    # documents: as if each were a sequence of its own
    first = np.repeat([0, 20], [2, 10]).astype(np.int32)
    docs = case.shaped(0.1, first=first)[0]
    alone = scored_ref.extend(case.q[2:], case.cache, case.tables, [30], [0, 10], 0.1, window=0, first=first[2:])[0]
    np.testing.assert_allclose(docs[2:], alone)
    np.testing.assert_allclose(docs[2], step_ref.extend(case.q[2:3], case.cache, case.tables, [21], [0, 1], 0.1, window=1)[0][0])
    # a span of one position is that position's value; an empty one gives zero
    one = case.shaped(0.1, first=np.full(12, 25, np.int32), last=np.full(12, 25, np.int32))[0]
    np.testing.assert_allclose(one[:, 0], np.broadcast_to(k[25], (12, 64)))
    assert not case.shaped(0.1, first=np.full(12, 25, np.int32), last=np.full(12, 24, np.int32))[0].any()


def test_documents_helper():
    rng = np.random.default_rng(3)
    first, last = scored_ref.documents(rng, [50, 0, 7], [50, 4, 100], 9, prefix=4)
    pos = np.concatenate([np.arange(50), np.arange(93, 100)])
    assert (first <= pos).all() and (pos <= last).all() and (pos - first < 9).all() and (last - first < 9).all()


# ------------------------------------------------------------------ refusals

def _norm(lib, desc=None, n=4, hq=4, q=FAKE, qo=FAKE + (1 << 24), qs=4 * 128, ks=256, rot=128, eps=1e-6, offset=0.0, qw=FAKE, kw=FAKE, key=FAKE, layer=0):
    return lib.pa_norm_rope_reshape_and_cache(V(qo), qs, V(q), qs, hq, V(), desc or _desc(), layer, V(key), ks, V(), 256, V(), V(), 0, V(), 100, rot, None, 1, 0,
                                              V(qw), V(kw), offset, eps, n, None, None)


def test_norm_refusals(lib):
    bad, unsup = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == bad, eps
    assert b"eps" in lib.pa_last_error_message()
    for offset in (float("nan"), float("inf")):
        assert _norm(lib, offset=offset) == bad, offset
    assert _norm(lib, qw=FAKE + 1) == bad and _norm(lib, kw=FAKE + 1) == bad
    assert b"k_weight" in lib.pa_last_error_message()
    # those of the call without norms
    assert _norm(lib, desc=_desc(head_size=96)) == unsup and _norm(lib, layer=1) == bad and _norm(lib, rot=24) == bad
    assert _norm(lib, key=0) == bad and _norm(lib, qs=4 * 128 - 8) == bad and _norm(lib, qo=FAKE + 16) == bad and _norm(lib, n=-1) == bad
    assert _norm(lib, n=0) == _lib.PA_OK


def _extend(lib, desc=None, S=2, T=100, Hq=4, max_q=100, q=FAKE, out=FAKE + (1 << 24), scale=0.1, window=0, ring=0, stride=8, width=8, cap=0.0, slopes=FAKE,
            first=FAKE, last=FAKE, ws=FAKE, ws_bytes=1 << 40, ctx=FAKE, qsl=FAKE):
    return lib.pa_extend_scored(V(out), V(q), Hq * 128, V(), desc or _desc(), 0, V(), stride, width, V(ctx), V(qsl), S, T, Hq, max_q, scale, window, ring, cap,
                                V(slopes), V(first), V(last), V(ws), ws_bytes, None, None)


def _decode(lib, desc=None, S=2, Hq=4, max_ctx=9000, q=FAKE, out=FAKE + (1 << 24), scale=0.1, window=0, ring=0, stride=8, width=8, cap=0.0, slopes=FAKE,
            first=FAKE, ws=FAKE, ws_bytes=1 << 40, ctx=FAKE):
    return lib.pa_decode_scored(V(out), V(q), Hq * 128, V(), desc or _desc(), 0, V(), stride, width, V(ctx), S, Hq, max_ctx, scale, window, ring, cap, V(slopes),
                                V(first), V(ws), ws_bytes, None, None)


@pytest.mark.parametrize("call", [_extend, _decode])
def test_scored_refusals(lib, call):
    bad, unsup = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
    for cap in (-1.0, float("nan"), float("inf"), 1e-5, 1e7):
        assert call(lib, cap=cap) == bad, cap
    assert b"softcap" in lib.pa_last_error_message()
    assert call(lib, slopes=FAKE + 2) == bad and call(lib, first=FAKE + 1) == bad
    assert call(lib, Hq=3) == bad and call(lib, Hq=34) == unsup and call(lib, desc=_desc(head_size=96)) == unsup
    assert call(lib, S=-1) == bad and call(lib, scale=0.0) == bad and call(lib, scale=float("nan")) == bad
    assert call(lib, window=-1) == bad and call(lib, ring=9) == bad and call(lib, stride=0) == bad and call(lib, width=9) == bad
    assert call(lib, q=0) == bad and call(lib, out=0) == bad and call(lib, ctx=0) == bad and call(lib, q=FAKE + 8) == bad
    assert call(lib, out=FAKE) == bad
    assert b"overlap" in lib.pa_last_error_message()
    assert call(lib, ws_bytes=100) == _lib.PA_ERR_WORKSPACE_TOO_SMALL and call(lib, ws=0) == bad
    assert call(lib, S=0) == _lib.PA_OK


def test_scored_refusals_of_their_own(lib):
    bad = _lib.PA_ERR_INVALID_ARG
    assert _extend(lib, last=FAKE + 2) == bad and _extend(lib, qsl=0) == bad and _extend(lib, max_q=-1) == bad
    assert _extend(lib, max_q=0) == _lib.PA_OK and _extend(lib, T=0) == _lib.PA_OK
    assert _decode(lib, max_ctx=0) == bad and _decode(lib, max_ctx=-5) == bad


def test_workspaces(lib):
    d = CacheDesc(16, 16, 2, 128, torch.bfloat16)
    assert _lib.extend_scored_workspace_bytes(d, 4, 100, 8, 50) >= _lib.extend_workspace_bytes(d, 4, 100, 8, 50) > 0
    assert _lib.decode_scored_workspace_bytes(d, 4, 8, 9000) == _lib.decode_workspace_bytes(d, 4, 8, 9000) > 0      # the decode kernel
    odd = CacheDesc(16, 16, 2, 128, torch.bfloat16)
    assert _lib.decode_scored_workspace_bytes(odd, 4, 6, 9000) == _lib.extend_scored_workspace_bytes(odd, 4, 4, 6, 1) > 0
    for args in ((0, 8, 100), (4, 0, 100), (4, 8, 0), (4, 9, 100), (4, 34, 100)):
        assert _lib.decode_scored_workspace_bytes(d, *args) == 0
    assert _lib.extend_scored_workspace_bytes(d, 4, 100, 8, 0) == 0


def test_binding_refuses_wrong_tensors():
    d = CacheDesc(4, 16, 2, 128, torch.float16)
    q = torch.zeros(3, 4, 128, dtype=torch.float16)
    kv = torch.zeros(3, 2, 128, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(*s)
    w = torch.zeros(128, dtype=torch.float16)

    def refused(fn, a, **kw):
        a = dict(a, **kw)
        with pytest.raises(_lib.PagedKVError) as e:
            fn(**a)
        assert e.value.status == _lib.PA_ERR_INVALID_ARG

    norm = dict(q_out=q, q=q, kv_cache=kv, desc=d, key=kv, value=kv, slot_mapping=torch.zeros(3, dtype=torch.int64), positions=i32(3),
                cos_sin=torch.zeros(10, 128), q_weight=w, k_weight=w, eps=1e-6)
    for bad in (w.float(), w[:64], torch.zeros(256, dtype=torch.float16)[::2], w[None]):
        refused(_lib.norm_rope_reshape_and_cache, norm, q_weight=bad)
        refused(_lib.norm_rope_reshape_and_cache, norm, k_weight=bad)
    refused(_lib.norm_rope_reshape_and_cache, norm, key=kv.bfloat16())
    refused(_lib.norm_rope_reshape_and_cache, norm, q=None, positions=i32(3).long())

    extend = dict(out=torch.zeros_like(q), q=q, kv_cache=kv, desc=d, block_tables=i32(1, 4), context_lens=i32(1), query_start_loc=i32(2), max_query_len=3, scale=0.1,
                  workspace=None)
    decode = dict(out=torch.zeros_like(q), q=q, kv_cache=kv, desc=d, block_tables=i32(3, 4), context_lens=i32(3), max_context_len=64, scale=0.1, workspace=None)
    for fn, a in ((_lib.extend_scored, extend), (_lib.decode_scored, decode)):
        refused(fn, a, q=q.bfloat16())
        refused(fn, a, out=q[:2])
        refused(fn, a, slopes=f32(4).double())
        refused(fn, a, slopes=f32(3))
        refused(fn, a, slopes=f32(8)[::2])
        refused(fn, a, first_pos=i32(3).long())
        refused(fn, a, first_pos=i32(2))
        refused(fn, a, first_pos=i32(6)[::2])
        refused(fn, a, block_tables=i32(4, 3).t())
        refused(fn, a, context_lens=a["context_lens"].long())
        refused(fn, a, q=q[:, :, :64], out=q[:, :, :64])
    refused(_lib.extend_scored, extend, last_pos=i32(4))
    refused(_lib.extend_scored, extend, last_pos=f32(3))
    refused(_lib.extend_scored, extend, query_start_loc=i32(1))
    refused(_lib.extend_scored, extend, query_start_loc=i32(2).long())
    refused(_lib.decode_scored, decode, context_lens=i32(2), block_tables=i32(2, 4))      # three queries, two sequences
    refused(_lib.decode_scored, decode, block_tables=i32(2, 4))


@pytest.mark.parametrize("name,to", [("fit", 1.0), ("near", 0.75)])
@pytest.mark.parametrize("cap", [30.0, 50.0, 1e6])
def test_cap_polynomials(cap, name, to):
    """The kernels' polynomials, in fp32 on the CPU, against tanh in 64 bits: within the bound that the tests use."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(_lib.__file__), "csrc", "extend_scored.cu")).read()
    fit = np.array([float(x) for x in re.search(r"%s\[\d\] = \{([^}]*)\}" % name, src).group(1).split(",")])
    y = np.linspace(-to, to, 200001).astype(np.float32)
    s = y * y
    coef = (fit * np.float32(cap)).astype(np.float32)
    v = np.full_like(y, coef[-1])
    for k in range(len(coef) - 2, -1, -1):
        v = (v * s).astype(np.float32) + coef[k]
    want = cap * np.tanh(y.astype(np.float64))
    assert (np.abs((v * y).astype(np.float64) - want) <= 2.0 ** -20 * np.abs(want)).all()
