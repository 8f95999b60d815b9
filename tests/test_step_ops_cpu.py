"""The serving-step operators without a GPU: their references against independent statements, and the
refusals of their entry points.  No call here reaches a kernel launch."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import step_ref
from paged_helpers import Paged, bits_to_f64, to_bits
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

@pytest.mark.parametrize("bs,D", [(1, 128), (2, 64), (8, 64), (16, 128), (32, 128)])
def test_layout_restated_agrees_with_the_oracle(bs, D):
    g = oracle.Geom(3, bs, 2, D, "f16")
    for part in range(2):
        got = step_ref.offsets16(bs, D, np.arange(bs), part)
        want = [[oracle.cache_offset(g, 0, 0, part, t, d) for d in range(D)] for t in range(bs)]
        assert np.array_equal(got, want)


@pytest.mark.parametrize("kv8", [False, True])
def test_cache_reads_what_the_oracle_wrote(kv8):
    rng = np.random.default_rng(0)
    c = step_ref.Cache(5, 4, 2, 128, "bf16", kv8)
    x = rng.standard_normal((2, 7, 2, 128))
    slots = rng.permutation(20)[:7]
    bits = [to_bits(y, "bf16") for y in x]
    assert c.write(bits[0], bits[1], slots) == 0
    for part in range(2):
        got, want = c.read(slots // 4, slots % 4, part), bits_to_f64(bits[part], "bf16")
        if kv8:   # half a code step of the vector's largest element
            assert (np.abs(got - want) <= np.abs(want).max(-1, keepdims=True) / 127 * 0.5001).all()
        else:
            assert np.array_equal(got, want)


def test_chunk_reference_of_single_tokens_is_decode():
    rng = np.random.default_rng(1)
    p = Paged(rng, S=3, Hq=6, Hkv=2, D=64, bs=8, ctx=[1, 20, 37], dtype="f16")
    c = step_ref.Cache(p.num_blocks, 8, 2, 64, "f16", False)
    c.pool = p.pool
    out, _ = step_ref.extend(p.q, c, p.tables, p.ctx, np.arange(4), 0.125)
    np.testing.assert_allclose(out, p.expected_contiguous(0.125), rtol=1e-12, atol=1e-14)


def test_rotations_agree_and_keep_lengths():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64))
    ang = rng.uniform(0, 100, (5, 16))
    for pairs in (False, True):
        y = step_ref.rotate64(x, ang, 32, pairs)
        y32 = step_ref.rotate32(x.astype(np.float32), np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32), 32, pairs)
        np.testing.assert_allclose(y32, y, atol=1e-5)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        # turning by a and then by b is turning by a + b
        np.testing.assert_allclose(step_ref.rotate64(y, ang, 32, pairs), step_ref.rotate64(x, 2 * ang, 32, pairs), atol=1e-12)


def test_table_reference_hands_out_blocks_like_the_block_manager(lib):
    # the host block manager gives out the highest free ids first, one request's blocks in logical order
    bm = _lib.BlockManager(4, 32)
    lens = [5, 1, 9]
    for s, n in enumerate(lens):
        bm.allocate(s, np.arange(n))
    free = np.arange(32, dtype=np.int32)
    qsl, ctx, slots, pos, tables, left, err = step_ref.build_tables(
        np.full((3, 4), -1, np.int32), free, 32, np.zeros(3, np.int32), np.asarray(lens, np.int32), 32, 4, 0, 15)
    assert err == 0 and left == bm.num_free()
    for s, n in enumerate(lens):
        t, _ = bm.block_table(s)
        assert tables[s, :len(t)].tolist() == t.tolist()
    bm.close()


# ------------------------------------------------------------------ refusals

def _rope(lib, desc=None, n=4, hq=4, q=FAKE, qo=FAKE, qs=4 * 128, qos=4 * 128, ks=256, rot=128, axes=1, pair_axis=None,
          axis_stride=0, maxpos=100, layer=0, key=FAKE, slots=FAKE, pos=FAKE, cs=FAKE):
    return lib.pa_rope_reshape_and_cache(V(qo), qos, V(q), qs, hq, V(), desc or _desc(), layer, V(key), ks, V(), 256,
                                         V(slots), V(pos), axis_stride, V(cs), maxpos, rot, pair_axis, axes, 0, n, None, None)


def test_rope_refusals(lib):
    bad, unsup = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
    assert _rope(lib, rot=24) == bad and _rope(lib, rot=0) == bad
    assert _rope(lib, rot=144) == bad                                       # more than head_size
    assert _rope(lib, axes=0) == bad and _rope(lib, axes=5) == bad
    assert _rope(lib, maxpos=0) == bad and _rope(lib, n=-1) == bad and _rope(lib, hq=-1) == bad
    assert _rope(lib, layer=1) == bad
    assert _rope(lib, desc=_desc(head_size=96)) == unsup
    assert _rope(lib, ks=248) == bad and _rope(lib, ks=260) == bad          # short, not a multiple of 8
    assert _rope(lib, qs=4 * 128 - 8) == bad and _rope(lib, qos=4 * 128 + 4) == bad
    assert _rope(lib, q=0) == bad and _rope(lib, q=FAKE + 8) == bad
    assert _rope(lib, key=0) == bad and _rope(lib, key=FAKE + 2) == bad
    assert _rope(lib, slots=FAKE + 4) == bad and _rope(lib, pos=FAKE + 2) == bad and _rope(lib, cs=FAKE + 1) == bad
    assert _rope(lib, axes=2, axis_stride=3) == bad                         # rows of positions overlap
    assert _rope(lib, axis_stride=-1) == bad
    # q_out overlapping q without being q
    assert _rope(lib, qo=FAKE + 16) == bad
    assert b"overlap" in lib.pa_last_error_message()
    assert _rope(lib, qos=8 * 128) == bad                                   # the same start, another stride
    axes = np.zeros(64, np.uint8)
    axes[63] = 3
    assert _rope(lib, axes=3, axis_stride=4, pair_axis=axes.ctypes.data) == bad
    assert b"pair_axis[63]" in lib.pa_last_error_message()
    assert _rope(lib, n=0) == _lib.PA_OK                                    # nothing to do


def _tables(lib, desc=None, S=2, T=8, stride=4, ring=0, qsl=FAKE, ctx=FAKE, slots=FAKE, pos=FAKE, tables=FAKE, free=FAKE,
            nf=FAKE, nfo=FAKE, cached=FAKE, new=FAKE):
    return lib.pa_build_tables(V(qsl), V(ctx), V(slots), V(pos), V(tables), stride, V(free), V(nf), V(nfo), desc or _desc(),
                               V(cached), V(new), S, T, ring, None, None)


def test_build_tables_refusals(lib):
    bad, unsup = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
    assert _tables(lib, S=-1) == bad and _tables(lib, T=-1) == bad
    assert _tables(lib, S=16385) == unsup
    assert _tables(lib, desc=_desc(block_size=12)) == unsup
    for name in ("qsl", "ctx", "slots", "tables", "free", "nf", "nfo", "cached", "new"):
        assert _tables(lib, **{name: 0}) == bad, name
    for name in ("qsl", "ctx", "pos", "tables", "free", "nf", "nfo", "cached", "new"):
        assert _tables(lib, **{name: FAKE + 2}) == bad, name
    assert _tables(lib, slots=FAKE + 4) == bad
    assert _tables(lib, stride=0) == bad
    assert _tables(lib, ring=5) == bad and _tables(lib, ring=-1) == bad     # a ring longer than its row


def _extend(lib, desc=None, S=2, T=100, Hq=4, max_q=100, q=FAKE, out=FAKE, scale=0.1, q_stride=None, window=0, ring=0, stride=8,
            ws=FAKE, ws_bytes=1 << 40, layer=0, ctx=FAKE, qsl=FAKE, bt=FAKE):
    return lib.pa_extend(V(out), V(q), Hq * 128 if q_stride is None else q_stride, V(), desc or _desc(), layer, V(bt), stride,
                         V(ctx), V(qsl), S, T, Hq, max_q, scale, window, ring, V(ws), ws_bytes, None, None)


def test_extend_refusals(lib):
    bad, unsup = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
    assert _extend(lib, Hq=3) == bad                                        # not a multiple of Hkv
    assert _extend(lib, Hq=34) == unsup                                     # group 17
    assert _extend(lib, desc=_desc(head_size=96)) == unsup
    assert _extend(lib, desc=_desc(kv_int8=True, head_size=64)) == unsup
    assert _extend(lib, layer=1) == bad and _extend(lib, S=-1) == bad and _extend(lib, S=70000) == bad
    assert _extend(lib, T=-1) == bad and _extend(lib, max_q=-1) == bad
    assert _extend(lib, scale=0.0) == bad and _extend(lib, scale=float("nan")) == bad
    assert _extend(lib, window=-1) == bad and _extend(lib, ring=-1) == bad and _extend(lib, ring=9) == bad
    assert _extend(lib, stride=0) == bad
    assert _extend(lib, q_stride=4 * 128 - 8) == bad and _extend(lib, q_stride=4 * 128 + 4) == bad
    for name in ("q", "out", "ctx", "qsl", "bt"):
        assert _extend(lib, **{name: 0}) == bad, name
    assert _extend(lib, q=FAKE + 8) == bad and _extend(lib, out=FAKE + 8) == bad
    assert _extend(lib, ctx=FAKE + 2) == bad and _extend(lib, qsl=FAKE + 1) == bad and _extend(lib, bt=FAKE + 2) == bad
    # out over q's first or last row
    q_bytes = 100 * 4 * 128 * 2
    assert _extend(lib) == bad and _extend(lib, out=FAKE + q_bytes - 16) == bad and _extend(lib, q=FAKE + q_bytes, out=FAKE + 16) == bad
    # nothing to do
    assert _extend(lib, S=0) == _lib.PA_OK and _extend(lib, T=0) == _lib.PA_OK and _extend(lib, max_q=0) == _lib.PA_OK


def test_binding_refuses_wrong_tensors():
    d = CacheDesc(4, 16, 2, 128, torch.float16)
    q = torch.zeros(3, 4, 128, dtype=torch.float16)
    kv = torch.zeros(3, 2, 128, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    slots, pos, cs = torch.zeros(3, dtype=torch.int64), i32(3), torch.zeros(10, 128)

    def rope(**kw):
        a = dict(q_out=q, q=q, kv_cache=kv, desc=d, key=kv, value=kv, slot_mapping=slots, positions=pos, cos_sin=cs)
        a.update(kw)
        with pytest.raises(_lib.PagedKVError) as e:
            _lib.rope_reshape_and_cache(**a)
        assert e.value.status == _lib.PA_ERR_INVALID_ARG

    rope(key=kv.bfloat16())
    rope(key=kv[:, :1])                                                     # too few kv heads
    rope(slot_mapping=i32(3))
    rope(positions=pos.long())
    rope(cos_sin=cs.double())
    rope(q=q[:, :, :64], q_out=q[:, :, :64])
    rope(q=q.transpose(0, 1).contiguous().transpose(0, 1))                  # heads not next to each other
    rope(pair_axis=np.zeros(3, np.uint8))

    def tables(**kw):
        a = dict(query_start_loc=i32(3), context_lens=i32(2), slot_mapping=slots, positions=i32(3), block_tables=i32(2, 4),
                 free_blocks=i32(4), num_free=i32(1), num_free_out=i32(1), desc=d, cached_lens=i32(2), new_lens=i32(2))
        a.update(kw)
        with pytest.raises(_lib.PagedKVError) as e:
            _lib.build_tables(**a)
        assert e.value.status == _lib.PA_ERR_INVALID_ARG

    tables(query_start_loc=i32(2))
    tables(free_blocks=i32(3))
    tables(positions=i32(2))
    tables(cached_lens=i32(2).long())
    tables(slot_mapping=i32(3))
    tables(block_tables=i32(4, 2).t())

    def extend(**kw):
        a = dict(out=q, q=q, kv_cache=kv, desc=d, block_tables=i32(1, 4), context_lens=i32(1), query_start_loc=i32(2),
                 max_query_len=3, scale=0.1, workspace=None)
        a.update(kw)
        with pytest.raises(_lib.PagedKVError) as e:
            _lib.extend(**a)
        assert e.value.status == _lib.PA_ERR_INVALID_ARG

    extend(q=q.bfloat16())
    extend(out=q[:2])
    extend(query_start_loc=i32(1))
    extend(context_lens=i32(1).long())
    extend(block_tables=i32(4, 2).t()[:1])                                 # entries two apart


def test_a_used_descriptor_is_copied_and_pickled_like_a_new_one():
    """A descriptor goes to worker processes; what a call keeps beside its fields does not."""
    import copy
    import dataclasses
    import pickle
    for used in (lambda d: d.c(), lambda d: d.ref(), _lib.cache_bytes):
        d = CacheDesc(4, 16, 2, 128, torch.bfloat16, num_layers=3, kv_int8=True)
        fields = dict(vars(d))
        size = _lib.cache_bytes(CacheDesc(**fields))
        used(d)
        assert vars(d) == fields == dataclasses.asdict(d)
        for e in (pickle.loads(pickle.dumps(d)), copy.copy(d), copy.deepcopy(d), CacheDesc(**vars(d)), dataclasses.replace(d)):
            assert e == d and _lib.cache_bytes(e) == size
            e.num_blocks = 8                                            # a copy's changes are its own
            assert e.c().num_blocks == 8 and d.c().num_blocks == 4 and _lib.cache_bytes(e) == 2 * size
        for protocol in range(pickle.HIGHEST_PROTOCOL + 1):
            assert pickle.loads(pickle.dumps(d, protocol)) == d


def test_rows_of_wider_tables_refusals(lib):
    bad = _lib.PA_ERR_INVALID_ARG

    def tables(stride, width, ring=0):
        return lib.pa_build_tables_strided(V(), V(), V(), V(), V(), stride, width, V(), V(), V(), _desc(), V(), V(), 2, 8, ring, None, None)

    def extend(stride, width, ring=0):
        return lib.pa_extend_strided(V(FAKE + (1 << 24)), V(), 512, V(), _desc(), 0, V(), stride, width, V(), V(), 2, 100, 4, 100, 0.1, 0,
                                     ring, V(), 1 << 40, None, None)
    for f in (tables, extend):
        assert f(8, 9) == bad and f(0, 0) == bad and f(8, -1) == bad and f(-8, -8) == bad
        assert f(8, 5, 6) == bad                                            # a ring longer than the width
        assert b"ring_blocks 6" in lib.pa_last_error_message()


def test_rows_share_memory_only_where_they_do(tmp_path):
    """The check of overlaps against every byte of drawn rows."""
    import os
    import shutil
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "rows_check")
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(os.path.dirname(here), "paged_kv_cache_168_gb300", "csrc"), os.path.join(here, "rows_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_outputs_over_inputs_are_refused(lib):
    bad = _lib.PA_ERR_INVALID_ARG
    A = FAKE

    def rope(q, qo, k, v, stride, n=4):                                     # 4 + 2 + 2 heads of 128: 1024, 512, 512 bytes
        r = lib.pa_rope_reshape_and_cache(V(A + qo), stride, V(A + q), stride, 4, V(), _desc(), 0, V(A + k), stride, V(A + v), stride, V(), V(), 0,
                                          V(), 100, 128, None, 1, 0, n, None, None)
        return r, lib.pa_last_error_message()
    # rows 4096 bytes apart: q_out over value's part, over key's, over the next row's key; 2048 bytes apart and in
    # place: over key; over half of q
    for args in ((0, 1536, 1024, 2048, 2048), (0, 1024, 1920, 3584, 2048), (512, 3584, 256, 2048, 2048), (0, 0, 512, 1536, 1024),
                 (0, 512, 2048, 3584, 2048)):
        r, msg = rope(*args)
        assert r == bad and b"overlap" in msg, (args, msg)

    def extend(q, out, stride):
        return lib.pa_extend(V(A + out), V(A + q), stride, V(), _desc(), 0, V(), 8, V(), V(), 2, 2, 4, 100, 0.1, 0, 0, V(), 0, None, None)
    small = _lib.PA_ERR_WORKSPACE_TOO_SMALL                                  # (checked after the overlap)
    # two rows of 1024 bytes: out (dense) between q's rows, over one, behind and before both
    assert extend(0, 1024, 4096) == small and extend(0, 2048, 2048) == small
    assert extend(0, 2064, 2048) == bad and extend(0, 1008, 4096) == bad and extend(0, 1024, 512) == bad
    assert extend(0, 2048, 512) == small and extend(2048, 0, 512) == small


@pytest.mark.parametrize("bad", [256, -1, 3, -256])
def test_axes_that_do_not_fit_a_byte_are_refused(bad):
    """An axis of 256 is not axis 0."""
    d = CacheDesc(4, 16, 2, 128, torch.float16)
    kv = torch.zeros(3, 2, 128, dtype=torch.float16)
    axes = np.zeros(64, np.int64)
    axes[5] = bad
    for pair_axis in (axes, axes.tolist(), torch.from_numpy(axes)):
        with pytest.raises(_lib.PagedKVError) as e:
            _lib.rope_reshape_and_cache(None, None, kv, d, kv, kv, torch.zeros(3, dtype=torch.int64), torch.zeros(3, 3, dtype=torch.int32),
                                        torch.zeros(10, 128), pair_axis=pair_axis)
        assert e.value.status == _lib.PA_ERR_INVALID_ARG
