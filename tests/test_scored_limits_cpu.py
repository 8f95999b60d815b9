"""Refusals and workspaces of the calls with shaped scores and normed heads at the ends of their ranges.  No call here
reaches a kernel launch."""
import pytest
import torch

from paged_kv_cache_168_gb300 import _lib, build as build_mod
from paged_kv_cache_168_gb300._lib import CacheDesc
from test_scored_ops_cpu import FAKE, _decode, _desc, _extend, _norm


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def test_eps_near_the_end_of_fp32(lib):
    assert _norm(lib, eps=1.1e38) == _lib.PA_ERR_INVALID_ARG and b"eps" in lib.pa_last_error_message()
    assert _norm(lib, eps=1e38, n=0) == _lib.PA_OK and _norm(lib, eps=1.4e-45, n=0) == _lib.PA_OK


@pytest.mark.parametrize("call", [_extend, _decode])
def test_quotients_of_scale_and_cap_that_leave_fp32(lib, call):
    """scale / softcap is a factor of every score: it has to be a normal number."""
    bad = _lib.PA_ERR_INVALID_ARG
    for scale, cap in ((1e35, 1e-4), (1e-33, 1e6), (1e-38, 1.0)):
        assert call(lib, scale=scale, cap=cap) == bad, (scale, cap)
        assert b"softcap" in lib.pa_last_error_message()
        assert call(lib, scale=scale, cap=0.0, S=0) == _lib.PA_OK     # (uncapped)
    assert call(lib, scale=float("inf"), cap=1.0) == bad
    for scale, cap in ((1e34, 1.0), (1e-30, 1e6), (1e30, 1e-4)):
        assert call(lib, scale=scale, cap=cap, S=0) == _lib.PA_OK, (scale, cap)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("window,ring", [(0, 12), (1500, 0), (100, 12)])
@pytest.mark.parametrize("S,Hq", [(1, 8), (256, 64), (8, 6)])
def test_windowed_workspaces_of_single_tokens(lib, S, Hq, window, ring, kv8):
    """What a windowed or ring call needs is what its span needs, whatever the contexts' length; the whole context's
    workspace is enough too."""
    d = CacheDesc(16, 16, 2, 128, torch.bfloat16, kv_int8=kv8)
    args = lambda n, ws=FAKE: dict(desc=_desc(dtype=torch.bfloat16, kv_int8=kv8), S=S, Hq=Hq, window=window, ring=ring, stride=1 << 27, width=1 << 27,
                                   out=FAKE + (1 << 40), ws_bytes=n, ws=ws)
    for most in (1400, 20000, 2**31 - 1):
        span = _lib.decode_window_span(most, 16, window, ring)
        of_span, of_all = _lib.decode_scored_workspace_bytes(d, S, Hq, span), _lib.decode_scored_workspace_bytes(d, S, Hq, most)
        if of_span == 0:                                             # (nothing left to refuse: the call would be made)
            continue
        for n in (of_span, of_all):                                  # refused for its address alone: the size is enough
            assert _decode(lib, max_ctx=most, **args(n, FAKE + 8)) == _lib.PA_ERR_INVALID_ARG, (most, n)
            assert b"aligned" in lib.pa_last_error_message()
        assert _decode(lib, max_ctx=most, **args(15)) == _lib.PA_ERR_WORKSPACE_TOO_SMALL
