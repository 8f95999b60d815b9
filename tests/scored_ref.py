"""Plain references of the operators of layers with normed heads and shaped scores, in numpy and 64 bits, with
bounds derived from the kernels' roundings.  Nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np

import step_ref
from step_ref import EPS, Chunk, attended_from


# ------------------------------------------------------------------ norms
def normed(x, weight, offset, eps):
    """x [.., D] float64 over its root mean square, times weight + offset (weight None: 1)."""
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return n if weight is None else n * (weight + offset)


def pair_sizes(x, rot, pairs):
    """|x1| + |x2| of every element's rotary pair (twice |x| of elements that are not turned)."""
    y = 2 * np.abs(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y


# Roundings before the result's own, in half-steps of fp32 relative to the pair's sizes: the sum of D squares as
# chains of 16 and up to four additions (20, half of it behind the root), the mean and eps (2), 1 / sqrt within two
# steps (4), weight + offset (1), two products (2); then cos and sin (2) and the rotation's (3).
NORM_STEPS = 24


# ------------------------------------------------------------------ attention with shaped scores
def spans(ctx, q_len, bs, window, ring, first, last):
    """[first, last] of a sequence's q_len newest positions; first, last: its tokens' entries or None."""
    out = []
    for j in range(q_len):
        pos = ctx - q_len + j
        a = attended_from(ctx, pos, bs, window, ring)
        if first is not None:
            a = max(a, int(first[j]))
        out.append((a, pos if last is None else min(int(last[j]), ctx - 1)))
    return out


def extend(q, cache, tables, ctx, qsl, scale, window=0, ring=0, cap=0.0, slopes=None, first=None, last=None):
    """q [T, Hq, D] float64 -> (out, tol) [T, Hq, D].

    tol as in step_ref.extend, with the errors of a token's shaped score s' weighted by the token:
      scores      ds_t = D 2^-22 scale sum |q k_t|, which a cap does not enlarge (its slope is at most 1);
      cap         2^-20 |c tanh(s / c)|: the polynomial is within 2^-20.7 of it and evaluated in fp32 (y = s / c and
                  six steps that at most double 2^-24 each); past |y| = 1, 2 / (1 + e^(2y)) <= 0.24 with relative
                  errors of 2^-22 of 2^x, 2^-24 of the sum and 2^-22 of the quotient, beside tanh >= 0.76;
      distance    2^-22 (slope (distance + 128) + |s'|): four roundings of fp32 of products and sums no larger than
                  the bias at a tile's first column, and of the slope in base 2;
    each changes the row by at most 2 sum_t p_t ds_t (|v_t| + |o|).
    """
    T, Hq, D = q.shape
    G = Hq // cache.Hkv
    u = EPS[cache.dtype] / 2
    u_p = EPS["f16"] / 2 if cache.kv8 else u
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    sl = np.zeros(Hq) if slopes is None else np.asarray(slopes, np.float64)
    sl = sl.reshape(cache.Hkv, G, 1)
    for s in range(len(ctx)):
        a, e, c = int(qsl[s]), int(qsl[s + 1]), int(ctx[s])
        if a == e:
            continue
        sp = spans(c, e - a, cache.bs, window, ring, None if first is None else first[a:e], None if last is None else last[a:e])
        some = [x for x in sp if x[0] <= x[1]]
        if not some:
            continue
        lo, end = min(x[0] for x in some), max(x[1] for x in some) + 1
        t = np.arange(lo, end)
        blk = t // cache.bs
        ids = tables[s, blk % ring if ring else blk]
        k, v = cache.read(ids, t % cache.bs, 0), cache.read(ids, t % cache.bs, 1)
        sv = cache.scales(ids, t % cache.bs, 1) if cache.kv8 else None
        for j, (f, g) in enumerate(sp):
            if f > g:
                continue
            pos = c - (e - a) + j
            kk, vv = k[f - lo:g + 1 - lo].transpose(1, 2, 0), v[f - lo:g + 1 - lo].transpose(1, 0, 2)
            qq = q[a + j].reshape(cache.Hkv, G, D)
            z = qq @ kk * scale                                        # [Hkv, G, n]
            ds = D * 2.0 ** -22 * scale * (np.abs(qq) @ np.abs(kk))
            if cap:
                z = cap * np.tanh(z / cap)
                ds = ds + 2.0 ** -20 * np.abs(z)
            far = np.abs(pos - np.arange(f, g + 1))
            if slopes is not None:
                ds = ds + 2.0 ** -22 * (np.abs(sl) * (far + 128) + np.abs(z))
                z = z - sl * far
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            with np.errstate(invalid="ignore"):                        # (infinities among the values)
                o, w = p @ vv, p @ np.abs(vv)
                moved = (p * ds) @ np.abs(vv) + (p * ds).sum(-1, keepdims=True) * np.abs(o)
            under = 2.0 ** -25 * np.abs(vv).sum(1)[:, None] if u_p == EPS["f16"] / 2 else 0.0
            if cache.kv8:
                ss = sv[f - lo:g + 1 - lo].T[:, :, None]               # [Hkv, n, 1]
                with np.errstate(invalid="ignore"):
                    codes = np.abs(vv) / np.where(ss > 0, ss, 1)
                under = 2.0 ** -21 * (ss.max(1) * codes.sum(1))[:, None]
            out[a + j] = o.reshape(Hq, D)
            tol[a + j] = (u * np.abs(o) + (u_p + 2.0 ** -16) * w + 2 * moved + under + 1e-30).reshape(Hq, D)
    return out, tol


def alibi(Hq):
    return (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)


def documents(rng, q_lens, ctx, longest, prefix=0, holes=0.0):
    """(first, last) of every query: documents of 1 to `longest` tokens, each with a prefix of up to `prefix` tokens
    that sees itself whole; a share `holes` of the queries sees nothing."""
    first, last = [], []
    for n, c in zip(np.asarray(q_lens).tolist(), np.asarray(ctx).tolist()):
        starts = np.concatenate([[0], np.cumsum(rng.integers(1, longest + 1, c + 1))])
        heads = rng.integers(0, prefix + 1, len(starts))
        p = np.arange(c - n, c)
        d = np.searchsorted(starts, p, side="right") - 1
        a = starts[d]
        b = np.maximum(p, np.minimum(a + heads[d], starts[d + 1]) - 1)
        first.append(np.where(rng.random(n) < holes, b + 1, a))
        last.append(b)
    return np.concatenate(first).astype(np.int32), np.concatenate(last).astype(np.int32)


class Scored(Chunk):
    """A chunk whose queries are `size` times as large: scores of that spread at scale 1 / sqrt(D)."""

    def __init__(self, rng, q_lens, ctx, size=1.0, **kw):
        super().__init__(rng, q_lens, ctx, **kw)
        if size != 1.0:
            self.q_bits = step_ref.to_bits(step_ref.bits_to_f64(self.q_bits, self.dtype) * size, self.dtype)
            self.q = step_ref.bits_to_f64(self.q_bits, self.dtype)

    def shaped(self, scale, window=0, **kw):
        return extend(self.q, self.cache, self.tables, self.ctx, self.qsl, scale, window, self.ring, **kw)
