"""The serving-step operators as a step uses them: lengths -> tables and slots -> rotary and cache write ->
attention of the new tokens, two steps in a row (prompts, then one chunk each), all on the device."""
import numpy as np
import pytest
import torch

import paged_kv_cache_168_gb300 as pkv
import step_ref
from gpu_helpers import dev_to_u16, ensure_built, u16_to_dev
from paged_helpers import bits_to_f64, to_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    ensure_built()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("window,bs", [(0, 16), (90, 16), (90, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_two_steps(kv8, window, bs, dtype):
    rng = np.random.default_rng(bs + window)
    S, Hq, Hkv, D, T = 4, 10, 2, 128, 400
    steps = [np.array([130, 1, 57, 0], np.int32), np.array([1, 100, 4, 33], np.int32)]
    ring = -(-(window + 130 - 1) // bs) + 1 if window else 0
    width = ring or 400 // bs
    nb = S * width + 5
    td = step_ref.torch_dtype(dtype)
    desc = pkv.CacheDesc(nb, bs, Hkv, D, td, kv_int8=kv8)
    pool = torch.zeros(pkv.cache_bytes(desc), dtype=torch.uint8, device="cuda")
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")
    tables, free = z(S, width) - 1, torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    nf = z(1) + nb
    lens, qsl, slots, pos, err = z(S), z(S + 1), z(T, dt=torch.int64), z(T), z(1)
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    table = pkv.rope_table(500, inv)
    scale = D ** -0.5
    K, V, held = [np.zeros((0, Hkv, D))] * S, [np.zeros((0, Hkv, D))] * S, np.zeros(S, int)
    ang = np.arange(500)[:, None] * inv.numpy()
    for new in steps:
        qb, kb, vb = (to_bits(rng.standard_normal((T, h, D)), dtype) for h in (Hq, Hkv, Hkv))
        q = u16_to_dev(qb, dtype)
        out = torch.full_like(q, 7.0)
        pkv.build_tables(qsl, lens, slots, pos, tables, free, nf, nf, desc, lens, torch.from_numpy(new).cuda(), ring_blocks=ring, dev_err=err)
        pkv.rope_reshape_and_cache(q, q, pool, desc, u16_to_dev(kb, dtype), u16_to_dev(vb, dtype), slots, pos, table, dev_err=err)
        ws = torch.empty(pkv.extend_workspace_bytes(desc, S, T, Hq, int(new.max())), dtype=torch.uint8, device="cuda")
        pkv.extend(out, q, pool, desc, tables, lens, qsl, int(new.max()), scale, ws, window=window, ring_blocks=ring, dev_err=err)
        assert pkv.read_device_errors(err) == 0
        n = int(new.sum())
        assert bool((out[n:] == 7).all()) and (slots[n:] == -1).all()
        # the same step without paging: rotated keys appended per sequence, attention over the last `window`
        at = 0
        for s in range(S):
            p = np.arange(held[s], held[s] + new[s])
            f = lambda bits: bits_to_f64(bits[at:at + new[s]], dtype)
            turn = lambda bits: step_ref.rotate64(f(bits), ang[p], D, False)
            K[s], V[s] = np.concatenate([K[s], turn(kb)]), np.concatenate([V[s], f(vb)])
            qq = turn(qb)
            held[s] += new[s]
            got = bits_to_f64(dev_to_u16(out[at:at + new[s]]), dtype)
            for j in range(new[s]):
                lo = max(0, p[j] - window + 1) if window else 0
                for h in range(Hq):
                    k, v = K[s][lo:p[j] + 1, h // 5], V[s][lo:p[j] + 1, h // 5]
                    w = np.exp((k @ qq[j, h]) * scale)
                    o = w @ v / w.sum()
                    # stored keys and queries are rounded once (u each), 8-bit codes are off by half a step of
                    # amax / 127; scores then move by ds, weights by 2 ds and again through their sum
                    u = step_ref.EPS[dtype] / 2
                    a, size = w / w.sum() @ np.abs(v), np.abs(qq[j, h])
                    code = (lambda x: np.abs(x).max(-1, keepdims=True) / 254) if kv8 else (lambda x: 0.0)
                    ds = scale * ((np.abs(k) * 2.01 * u + code(k)) @ size).max()
                    tol = u * np.abs(o) + (u + 4 * ds + 2.0 ** -12) * a + (code(v).max() if kv8 else 0.0) + 2.0 ** -25 * np.abs(v).sum(0)
                    assert (np.abs(got[j, h] - o) <= tol).all(), (s, j, h)
            at += new[s]
    # decode over the cache these steps left agrees with the chunk of one token
    dec = torch.empty((S, Hq, D), dtype=td, device="cuda")
    qd = u16_to_dev(to_bits(rng.standard_normal((S, Hq, D)), dtype), dtype)
    if Hq // Hkv == 5:                                                 # decode takes groups of 1, 2, 4, 8: take 4 of 5 heads
        qd = qd.unflatten(1, (Hkv, 5))[:, :, :4].reshape(S, 8, D).contiguous()
        dec = torch.empty_like(qd)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    pkv.decode_window(dec, qd, pool, desc, tables, lens, 400, scale, window, ring, ws, dev_err=err)
    one = torch.empty_like(qd)
    ones = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.extend_workspace_bytes(desc, S, S, 8, 1), dtype=torch.uint8, device="cuda")
    pkv.extend(one, qd, pool, desc, tables, lens, ones, 1, scale, ws, window=window, ring_blocks=ring, dev_err=err)
    assert pkv.read_device_errors(err) == 0
    # both round their output and their weights (u, and u of the weighted sizes: at most max |v| < 6)
    u = step_ref.EPS[dtype] / 2
    assert bool(((dec.double() - one.double()).abs() <= 2 * u * one.double().abs() + 2 * u * 6 + 1e-4).all())
