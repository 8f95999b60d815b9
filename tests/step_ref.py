"""Plain references of the serving-step operators (block tables from lengths,
rotary positions with the cache write, attention of a chunk over the cache), in
numpy: Python loops and 64-bit arithmetic where values are real, IEEE binary32
where the result is defined bit by bit.  Nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from paged_helpers import bits_to_f64, to_bits

EPS = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}      # torch.finfo(t).eps: a rounding is off by at most half of it


# ------------------------------------------------------------------ cache layout, restated
def chunk_elements(bs, D):
    return 2 * bs * D


def offsets16(bs, D, t, part):
    """Element offsets [len(t), D] inside a 16-bit chunk of slot t's vector."""
    t = np.asarray(t, np.int64)[:, None]
    d = np.arange(D)[None, :]
    R = min(bs, 8)
    g, r = t // R, t % R
    return ((g * 2 + part) * (D // 64) + d // 64) * (R * 64) + r * 64 + (((d % 64) // 8) ^ r) * 8 + d % 8


def scale_bytes(bs):
    return (4 * bs + 15) // 16 * 16


def chunk_bytes8(bs):
    return 2 * bs * 128 + 2 * scale_bytes(bs)


def offsets8(bs, t, part):
    """Byte offsets [len(t), 128] inside an 8-bit chunk of slot t's codes."""
    t = np.asarray(t, np.int64)[:, None]
    d = np.arange(128)[None, :]
    return (part * bs + t) * 128 + (((d // 16) ^ (t % 8)) * 16) + d % 16


class Cache:
    """A pool as numpy, its geometry, and reads of it as float64."""

    def __init__(self, num_blocks, bs, Hkv, D, dtype, kv8, fill_nan=True):
        self.nb, self.bs, self.Hkv, self.D, self.dtype, self.kv8 = num_blocks, bs, Hkv, D, dtype, kv8
        if kv8:
            self.pool = np.zeros(num_blocks * Hkv * chunk_bytes8(bs), np.uint8)
        else:
            nan = {"f16": 0x7E00, "bf16": 0x7FC0}[dtype]
            self.pool = np.full(num_blocks * Hkv * chunk_elements(bs, D), nan if fill_nan else 0, np.uint16)

    def geom(self):
        return oracle.Geom(self.nb, self.bs, self.Hkv, self.D, self.dtype)

    def write(self, key_bits, value_bits, slots):
        f = oracle.reshape_and_cache_i8 if self.kv8 else oracle.reshape_and_cache
        return f(self.pool, self.geom(), key_bits, value_bits, np.asarray(slots, np.int64))

    def read(self, block, t, part):
        """[n, Hkv, D] float64 of slots (block[i], t[i])."""
        block, t = np.asarray(block, np.int64), np.asarray(t, np.int64)
        out = np.empty((len(t), self.Hkv, self.D))
        for h in range(self.Hkv):
            if self.kv8:
                base = (block * self.Hkv + h) * chunk_bytes8(self.bs)
                codes = self.pool[base[:, None] + offsets8(self.bs, t, part)].view(np.int8).astype(np.float64)
                so = base + 2 * self.bs * 128 + part * scale_bytes(self.bs) + 4 * t
                out[:, h] = codes * self.pool.view(np.float32)[so // 4].astype(np.float64)[:, None]
            else:
                base = (block * self.Hkv + h) * chunk_elements(self.bs, self.D)
                out[:, h] = bits_to_f64(self.pool[base[:, None] + offsets16(self.bs, self.D, t, part)], self.dtype)
        return out


    def scales(self, block, t, part):
        """[n, Hkv] float64 scales of slots (8-bit caches)."""
        block, t = np.asarray(block, np.int64), np.asarray(t, np.int64)
        at = [((block * self.Hkv + h) * chunk_bytes8(self.bs) + 2 * self.bs * 128 + part * scale_bytes(self.bs) + 4 * t) // 4
              for h in range(self.Hkv)]
        return np.stack([self.pool.view(np.float32)[a] for a in at], 1).astype(np.float64)


# ------------------------------------------------------------------ block tables from lengths
OUT_OF_BLOCKS, CONTEXT, BLOCK_ID = 32, 4, 1


def build_tables(tables, free, num_free, cached, new, num_blocks, bs, ring, max_tokens):
    """(query_start_loc, context_lens, slots, positions, tables, num_free, error bits)."""
    S, width = tables.shape
    tables = tables.copy()
    R = ring or 1 << 60
    err = 0
    for c, n in zip(cached.tolist(), new.tolist()):
        if c < 0 or n < 0 or c + n > 2**31 - 1 or (not ring and c + n > width * bs):
            err |= CONTEXT
    blocks = lambda x: min(-(-x // bs), R)
    if not err:
        if int(new.astype(np.int64).sum()) > max_tokens:
            err |= CONTEXT
        took = sum(blocks(int(c) + int(n)) - blocks(int(c)) for c, n in zip(cached, new))
        if num_free < 0 or num_free > num_blocks or took > num_free:
            err |= OUT_OF_BLOCKS
    elif num_free < 0 or num_free > num_blocks:
        err |= OUT_OF_BLOCKS
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32)
    if err:
        return np.zeros(S + 1, np.int32), np.zeros(S, np.int32), slots, positions, tables, num_free, err
    at, qsl, ctx = 0, [0], []
    for s in range(S):
        c, n = int(cached[s]), int(new[s])
        for b in range(blocks(c), blocks(c + n)):
            num_free -= 1
            tables[s, b] = free[num_free]
        for pos in range(c, c + n):
            b = pos // bs
            positions[at] = pos
            if not ring or b > (c + n - 1) // bs - ring:
                block = int(tables[s, b % R])
                if 0 <= block < num_blocks:
                    slots[at] = block * bs + pos % bs
                else:
                    err |= BLOCK_ID
            at += 1
        qsl.append(at)
        ctx.append(c + n)
    return np.asarray(qsl, np.int32), np.asarray(ctx, np.int32), slots, positions, tables, num_free, err


# ------------------------------------------------------------------ rotary positions
def rotate32(x, cos, sin, rot, pairs):
    """x [N, H, D] float32; cos, sin [N, rot / 2] float32: binary32 products and sums, one rounding each."""
    y = x.astype(np.float32).copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2, c, s = x[..., a], x[..., b], cos[:, None], sin[:, None]
    y[..., a] = (x1 * c).astype(np.float32) - (x2 * s).astype(np.float32)
    y[..., b] = (x2 * c).astype(np.float32) + (x1 * s).astype(np.float32)
    return y


def rotate64(x, angles, rot, pairs):
    """x [N, H, D] float64; angles [N, rot / 2] float64: complex multiplication."""
    y = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angles)[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def quantise(x):
    """Codes and scale [.., 1] of float32 vectors [.., 128]: symmetric, binary32 throughout, products with
    reciprocals (127 * (1 / amax), amax * (1 / 127))."""
    one, n = np.float32(1), np.float32(127)
    amax = np.abs(x).max(-1, keepdims=True).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(amax > 0, n * (one / amax), np.float32(0)).astype(np.float32)
        inv = np.minimum(inv, np.finfo(np.float32).max)
        codes = np.clip(np.rint((x * inv).astype(np.float32)), -127, 127).astype(np.int8)
        return codes, (amax * (one / n)).astype(np.float32)


def store8(cache, codes, scales, part, slots):
    """Write codes [N, Hkv, 128] and scales [N, Hkv, 1] at slots (skipping -1) into an 8-bit pool."""
    for i, slot in enumerate(np.asarray(slots).tolist()):
        if slot == -1:
            continue
        block, t = slot // cache.bs, slot % cache.bs
        for h in range(cache.Hkv):
            base = (block * cache.Hkv + h) * chunk_bytes8(cache.bs)
            cache.pool[base + offsets8(cache.bs, [t], part)[0]] = codes[i, h].view(np.uint8)
            so = base + 2 * cache.bs * 128 + part * scale_bytes(cache.bs) + 4 * t
            cache.pool[so:so + 4] = scales[i, h].astype(np.float32).view(np.uint8)


# ------------------------------------------------------------------ attention of a chunk
def attended_from(ctx, pos, bs, window, ring):
    t = max(0, pos - window + 1) if window else 0
    return max(t, ((ctx - 1) // bs - ring + 1) * bs) if ring else t


def extend(q, cache, tables, ctx, qsl, scale, window=0, ring=0, num_tokens=None):
    """q [T, Hq, D] float64 -> (out, tol) [T, Hq, D].

    tol bounds |kernel - out| elementwise.  With u the half-step of the output's type,
    w = sum_t p_t |v_t| and the rounding of a weight at most u_p relative (u_p = u; for an 8-bit cache the
    weights are fp16):
      output rounding         u |o|
      weights' rounding       u_p w, plus 2^-25 sum_t |v_t| for fp16 weights below its normal range
                              (weights are taken against a running maximum, so the normaliser is at least 1);
                              weights of an 8-bit cache carry the token's scale s_t and are taken against
                              x + log2 of the largest scale or at most 16 times it (masked tokens'), so the
                              normaliser is at least 1 / (16 max s), and a stored weight meets the code
                              v_t / s_t: 16 2^-25 max s sum_t |v_t| / s_t
      scores                  D products summed in fp32, each step off by at most 2^-22 of the sum of the
                              terms' sizes (2^-23 rounded, twice that if truncated): ds = D 2^-22 scale
                              sum |q k|; a relative change of at most 2 ds of every weight, and again of
                              their sum: 4 ds w
      2^x, sums, rescaling    2^-16 w (a few ulps of fp32 for each of up to 2^17 / 128 tiles' sums)
    """
    T, Hq, D = q.shape
    G = Hq // cache.Hkv
    u = EPS[cache.dtype] / 2
    u_p = EPS["f16"] / 2 if cache.kv8 else u
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for s in range(len(ctx)):
        a, e, c = int(qsl[s]), int(qsl[s + 1]), int(ctx[s])
        if a == e:
            continue
        lo = min(attended_from(c, c - (e - a) + j, cache.bs, window, ring) for j in range(e - a))
        t = np.arange(lo, c)
        blk = t // cache.bs
        ids = tables[s, blk % ring if ring else blk]
        k, v = cache.read(ids, t % cache.bs, 0), cache.read(ids, t % cache.bs, 1)
        sv = cache.scales(ids, t % cache.bs, 1) if cache.kv8 else None
        for j in range(e - a):
            pos = c - (e - a) + j
            f = attended_from(c, pos, cache.bs, window, ring)
            if f > pos:
                continue
            kk, vv = k[f - lo:pos + 1 - lo].transpose(1, 2, 0), v[f - lo:pos + 1 - lo].transpose(1, 0, 2)
            qq = q[a + j].reshape(cache.Hkv, G, D)
            z = qq @ kk * scale                                        # [Hkv, G, n]
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            with np.errstate(invalid="ignore"):                        # (infinities among the values)
                o, w = p @ vv, p @ np.abs(vv)
            ds = D * 2.0 ** -22 * scale * (np.abs(qq) @ np.abs(kk)).max(-1, keepdims=True)
            under = 2.0 ** -25 * np.abs(vv).sum(1)[:, None] if u_p == EPS["f16"] / 2 else 0.0
            if cache.kv8:
                ss = sv[f - lo:pos + 1 - lo].T[:, :, None]             # [Hkv, n, 1]
                with np.errstate(invalid="ignore"):
                    codes = np.abs(vv) / np.where(ss > 0, ss, 1)
                under = 2.0 ** -21 * (ss.max(1) * codes.sum(1))[:, None]
            out[a + j] = o.reshape(Hq, D)
            tol[a + j] = (u * np.abs(o) + (u_p + 4 * ds + 2.0 ** -16) * w + under + 1e-30).reshape(Hq, D)
    return out, tol


class Chunk:
    """Sequences whose newest q_lens[s] of ctx[s] tokens are queries, over a pool written by the oracle (NaN in
    16-bit slots that hold nothing)."""

    def __init__(self, rng, q_lens, ctx, Hq, Hkv, D, bs, dtype, kv8=False, ring=0, scale_k=1.0, extra_rows=0):
        self.dtype, self.ring, self.Hq = dtype, ring, Hq
        self.q_lens, self.ctx = np.asarray(q_lens, np.int32), np.asarray(ctx, np.int32)
        S = len(self.ctx)
        nblk = np.minimum(-(-self.ctx // bs), ring or 1 << 30)
        width = ring or max(int(nblk.max()), 1)
        self.cache = Cache(int(nblk.sum()) + 3, bs, Hkv, D, dtype, kv8)
        perm = rng.permutation(self.cache.nb)
        self.tables = np.full((S, width), -1, np.int32)
        at = 0
        for s in range(S):
            self.tables[s, :nblk[s]] = perm[at:at + nblk[s]]
            at += int(nblk[s])
            c = int(self.ctx[s])
            if c == 0:
                continue
            t = np.arange(c)
            blk = t // bs
            slots = self.tables[s, blk % ring if ring else blk].astype(np.int64) * bs + t % bs
            k, v = rng.standard_normal((c, Hkv, D)) * scale_k, rng.standard_normal((c, Hkv, D))
            assert self.cache.write(to_bits(k, dtype), to_bits(v, dtype), slots) == 0
        self.qsl = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        self.T = int(self.qsl[-1]) + extra_rows
        self.q_bits = to_bits(rng.standard_normal((self.T, Hq, D)), dtype)
        self.q = bits_to_f64(self.q_bits, dtype)

    def expected(self, scale, window=0):
        return extend(self.q, self.cache, self.tables, self.ctx, self.qsl, scale, window, self.ring)


def torch_dtype(name):
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]
