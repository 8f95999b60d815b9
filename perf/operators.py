"""Cases and plain forms of the serving-step operators around the paged cache.

tables   block tables, slot maps and positions of a step, built from request lengths
rope     rotary positions with one or several axes on q and k, and the write of k and v into the cache
extend   attention of a chunk of new tokens per sequence over the paged cache

``own`` False: elementary torch operations in 32 bits.  ``own`` True: the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    T, R, E = "tables", "rope", "extend"
    return [
        # a decode step of 256 requests: one new token each
        dict(name="tables_decode", op=T, seqs=256, new_lo=1, new_hi=1, cached_lo=1, cached_hi=8191, bs=16, ring=0, pad=0),
        # sixteen prompts of 2048 tokens
        dict(name="tables_prompts", op=T, seqs=16, new_lo=2048, new_hi=2048, cached_lo=0, cached_hi=0, bs=16, ring=0, pad=0),
        # a large mixed batch over sliding-window ring tables, padded to a captured graph's token count
        dict(name="tables_ring", op=T, seqs=2000, new_lo=0, new_hi=61, cached_lo=0, cached_hi=9000, bs=32, ring=33, pad=999),
        # the new token of 256 decoding requests, grouped heads
        dict(name="rope_decode", op=R, tokens=256, hq=32, hkv=8, d=128, rot=128, bs=16, dtype="bf16", kv8=False, axes=1, pairs=False, cycle=False, far=8192),
        # a batch of video and image prompts: time, height and width
        dict(name="rope_video", op=R, tokens=32768, hq=32, hkv=8, d=128, rot=128, bs=16, dtype="bf16", kv8=False, axes=3, pairs=False, cycle=False, far=4096),
        # prompts into an 8-bit cache, half of each head rotated, neighbouring pairs, axes taken in turn
        dict(name="rope_int8", op=R, tokens=5001, hq=32, hkv=32, d=128, rot=64, bs=16, dtype="f16", kv8=True, axes=2, pairs=True, cycle=True, far=131072),
        # the smallest call: a handful of new tokens over short contexts, where latency counts
        dict(name="extend_tiny", op=E, seqs=4, q_lo=1, q_hi=5, pre_lo=0, pre_hi=95, hq=4, hkv=4, d=64, bs=16, dtype="f16", kv8=False, window=0, ring=False),
        # checking four drafted tokens a request against long contexts
        dict(name="extend_verify", op=E, seqs=8, q_lo=4, q_hi=4, pre_lo=32764, pre_hi=131068, hq=64, hkv=8, d=128, bs=32, dtype="bf16", kv8=False, window=0, ring=False),
        # chunked prefill: 512-token chunks over cached prefixes
        dict(name="extend_chunks", op=E, seqs=32, q_lo=512, q_hi=512, pre_lo=512, pre_hi=3584, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=False, window=0, ring=False),
        # whole prompts
        dict(name="extend_prompts", op=E, seqs=16, q_lo=2048, q_hi=2048, pre_lo=0, pre_hi=0, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=False, window=0, ring=False),
        # ragged chunks over an 8-bit cache
        dict(name="extend_int8", op=E, seqs=32, q_lo=1, q_hi=700, pre_lo=1, pre_hi=3500, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=True, window=0, ring=False),
        # a sliding window over ring tables, token-granular blocks, an odd number of heads a group
        dict(name="extend_window", op=E, seqs=13, q_lo=33, q_hi=301, pre_lo=100, pre_hi=6000, hq=10, hkv=2, d=128, bs=1, dtype="f16", kv8=False, window=1000, ring=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = (max(most.get(c["op"], (0, 0))[0], w["bytes"]), max(most.get(c["op"], (0, 0))[1], w["flops"]))
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1] and _plain_cost(c) <= 6e9:
            return c


def _plain_cost(c):
    # scores of the plain form's padded rectangle
    return c["seqs"] * c["hq"] * c["q_hi"] * (c["pre_hi"] + c["q_hi"]) if c["op"] == "extend" else 0


def _draw(rng):
    op = rng.choice(["tables", "rope", "extend", "extend"])
    if op == "tables":
        new_hi = _log(rng, 1, 2048)
        seqs = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, new_lo=rng.randint(0, new_hi), new_hi=new_hi, cached_lo=0, cached_hi=_log(rng, 1, 9000), bs=rng.choice([1, 2, 4, 8, 16, 32]),
                    ring=rng.choice([0, 0, rng.randint(3, 70)]), pad=rng.choice([0, rng.randint(1, 999)]))
    if op == "rope":
        d = rng.choice([64, 128])
        kv8 = d == 128 and rng.random() < 0.4
        hkv = rng.choice([1, 2, 4, 8, 32])
        return dict(op=op, tokens=_log(rng, 1, 32768), hq=hkv * rng.choice([1, 4, 5, 8]), hkv=hkv, d=d, rot=rng.choice([d, d // 2]), bs=rng.choice([1, 2, 4, 8, 16, 32]),
                    dtype=rng.choice(["f16", "bf16"]), kv8=kv8, axes=rng.randint(1, 3), pairs=rng.random() < 0.5, cycle=rng.random() < 0.5, far=_log(rng, 1024, 131072))
    d = rng.choice([64, 128, 128])
    kv8 = d == 128 and rng.random() < 0.4
    hkv = rng.choice([1, 2, 4, 8])
    q_hi = _log(rng, 1, 2048)
    pre_hi = _log(rng, 1, 131068) if q_hi < 9 else _log(rng, 1, 9000)
    window = rng.choice([0, 0, rng.randint(1, 2000)])
    return dict(op=op, seqs=_log(rng, 1, 64), q_lo=rng.randint(0 if q_hi > 1 else 1, q_hi), q_hi=q_hi, pre_lo=rng.randint(0, pre_hi), pre_hi=pre_hi,
                hq=hkv * rng.choice([1, 2, 4, 5, 8, 16]), hkv=hkv, d=d, bs=rng.choice([1, 4, 8, 16, 16, 32]), dtype=rng.choice(["f16", "bf16"]), kv8=kv8,
                window=window, ring=window > 0 and rng.random() < 0.5)


# ------------------------------------------------------------------ lengths (from the case and a seed, on the host)

def _lens(case, seed):
    """Lengths of a case's requests: tables (cached, new), extend (prefix, q_len).  A seed puts them in an order of its own."""
    g = np.random.default_rng(7)
    lo, hi, a, b = ("new_lo", "new_hi", "cached_lo", "cached_hi") if case["op"] == "tables" else ("q_lo", "q_hi", "pre_lo", "pre_hi")
    S = case["seqs"]
    new, old = g.integers(case[lo], case[hi] + 1, S), g.integers(case[a], case[b] + 1, S)
    if new.sum() == 0:
        new[-1] = max(1, case[hi])
    order = np.random.default_rng(seed & 0xFFFFFFFF).permutation(S)
    return old[order].astype(np.int64), new[order].astype(np.int64)


def _ring_blocks(case):
    # a ring that holds every window of a chunk exactly
    return -(-(case["window"] + case["q_hi"] - 1) // case["bs"]) + 1 if case["ring"] else 0


def _starts(case, old, new):
    """First attended position of each request's first query."""
    w = case["window"]
    return np.maximum(0, old - w + 1) if w else np.zeros_like(old)


def work(case):
    if case["op"] == "rope":
        T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        kv = 2 * hkv * (d + 4) if case["kv8"] else 4 * hkv * d
        return {"bytes": T * (4 * hq * d + 4 * hkv * d + kv + 4 * case["axes"] + 8), "flops": T * (hq + hkv) * case["rot"] * 3}
    old, new = _lens(case, 0)
    if case["op"] == "tables":
        S, T, bs = case["seqs"], int(new.sum()) + case["pad"], case["bs"]
        cap = case["ring"] or 1 << 30
        took = int((np.minimum(-(-(old + new) // bs), cap) - np.minimum(-(-old // bs), cap)).sum())
        return {"bytes": 8 * S + 4 * (S + 1) + 4 * S + 12 * T + 8 * took + 8, "flops": 0}
    d, hq, hkv, w = case["d"], case["hq"], case["hkv"], case["window"]
    ctx = old + new
    if w:
        full = np.array([np.minimum(np.arange(a, b) + 1, w).sum() for a, b in zip(old, ctx)])
    else:
        full = new * old + new * (new + 1) // 2
    kv = hkv * (2 * d + 8) if case["kv8"] else 4 * hkv * d
    span = int(((ctx - _starts(case, old, new)) * (new > 0)).sum())
    T = int(new.sum())
    return {"bytes": 4 * T * hq * d + span * kv + 4 * (span // case["bs"] + 2 * case["seqs"]), "flops": float(4 * d * hq * int(full.sum()))}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _pool(case, nb, g):
    """Cache memory of nb blocks that holds normal values (16-bit), or codes and scales (8-bit)."""
    hkv, bs, d = case["hkv"], case["bs"], case["d"]
    if not case["kv8"]:
        return torch.cat([_normal((min(4096, nb - i), hkv, 2 * bs * d), DTYPES[case["dtype"]], g) for i in range(0, nb, 4096)])
    sb = -(-4 * bs // 16) * 16
    pool = torch.zeros((nb, hkv, 2 * bs * d + 2 * sb), dtype=torch.uint8, device=DEV)
    x = torch.randn((nb, hkv, 2 * bs * d), generator=g, device=DEV).mul_(127 / 3.2).round_().clamp_(-127, 127)
    pool[..., :2 * bs * d] = x.to(torch.int8).view(torch.uint8)
    s = (torch.rand((nb, hkv, 2, sb // 4), generator=g, device=DEV) * 1.6 + 2.0) / 127
    pool[..., 2 * bs * d:] = s.view(nb, hkv, -1).view(torch.uint8)
    return pool


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    if op == "tables":
        return _prepare_tables(case, seed, g)
    return _prepare_rope(case, seed, g) if op == "rope" else _prepare_extend(case, seed, g)


def _prepare_tables(case, seed, g):
    old, new = _lens(case, seed)
    S, bs, cap = case["seqs"], case["bs"], case["ring"] or 1 << 30
    have = np.minimum(-(-old // bs), cap)
    need = np.minimum(-(-(old + new) // bs), cap)
    width = case["ring"] or int(max(need.max(), 1))
    nb = int(1.1 * need.sum()) + 8
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    h = torch.from_numpy(have).to(DEV)
    col = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(h, 0) - h)[:, None] + col
    tables = torch.where(col < h[:, None], perm[at.clamp(max=nb - 1)], torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous()
    n = nb - int(have.sum())
    free = torch.full((nb,), -1, dtype=torch.int32, device=DEV)
    free[:n] = perm[nb - n:]
    T = int(new.sum()) + case["pad"]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, cached=_i32(old), new=_i32(new), tables=tables, free=free, num_free=torch.tensor([n], **i32), num_blocks=nb,
                qsl=torch.empty(S + 1, **i32), ctx=torch.empty(S, **i32), slots=torch.empty(T, dtype=torch.int64, device=DEV),
                positions=torch.empty(T, **i32), left=torch.empty(1, **i32), err=torch.zeros(1, **i32))


def _pair_axis(case):
    n, a = case["rot"] // 2, case["axes"]
    return (np.arange(n) % a if case["cycle"] else np.arange(n) * a // n).astype(np.uint8)


def _prepare_rope(case, seed, g):
    T, hq, hkv, d, rot, bs = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot", "bs"))
    dt = DTYPES[case["dtype"]]
    nb = int(1.1 * T) // bs + 2
    far = case["far"]
    if case["axes"] == 1:
        pos = torch.randint(0, far, (1, T), generator=g, device=DEV, dtype=torch.int32)
    else:  # frames of a grid, row by row, from a place of their own
        i = torch.arange(T, device=DEV)
        start = int(torch.randint(0, max(1, far - T // 576 - 64), (1,), generator=g, device=DEV)[0])
        pos = torch.stack([(start + i // 576) % far, start + i // 24 % 24, start + i % 24][:case["axes"]]).to(torch.int32).contiguous()
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    ang = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * inv
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:T].contiguous()
    slots[torch.rand(T, generator=g, device=DEV) < 0.02] = -1  # padding, and tokens that the cache holds already
    q = _normal((T, hq, d), dt, g)
    return dict(case=case, q=q, q_out=torch.empty_like(q), key=_normal((T, hkv, d), dt, g), value=_normal((T, hkv, d), dt, g), pool=_pool(case, nb, g), num_blocks=nb,
                slots=slots, positions=pos, cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(), pair_axis=_pair_axis(case),
                err=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_extend(case, seed, g):
    old, new = _lens(case, seed)
    S, hq, d, bs = case["seqs"], case["hq"], case["d"], case["bs"]
    ctx, ring = old + new, _ring_blocks(case)
    nblk = np.minimum(-(-ctx // bs), ring or 1 << 30)
    width = ring or int(max(nblk.max(), 1))
    nb = int(1.05 * nblk.sum()) + 2
    h = torch.from_numpy(nblk).to(DEV)
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(h, 0) - h)[:, None] + col
    tables = torch.where(col < h[:, None], perm[at.clamp(max=nb - 1)], torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous()
    T = int(new.sum())
    q = _normal((T, hq, d), DTYPES[case["dtype"]], g)
    s = dict(case=case, q=q, out=torch.empty_like(q), pool=_pool(case, nb, g), num_blocks=nb, tables=tables, ctx=_i32(ctx), qsl=_i32(np.concatenate([[0], np.cumsum(new)])),
             max_q=int(new.max()), max_ctx=int(ctx.max()), ring=ring, scale=1 / math.sqrt(d), err=torch.zeros(1, dtype=torch.int32, device=DEV), ws=None)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own_tables(s) if op == "tables" else _own_rope(s) if op == "rope" else _own_extend(s)
    return _plain_tables(s) if op == "tables" else _plain_rope(s) if op == "rope" else _plain_extend(s)


def _desc(s):
    """The cache's geometry, which a user's program keeps beside its pool."""
    if "desc" not in s:
        import paged_kv_cache_168_gb300 as pkv
        c = s["case"]
        s["desc"] = pkv.CacheDesc(s["num_blocks"], c["bs"], 1, 128) if c["op"] == "tables" else \
            pkv.CacheDesc(s["num_blocks"], c["bs"], c["hkv"], c["d"], DTYPES[c["dtype"]], kv_int8=c["kv8"])
    return s["desc"]


def _own_tables(s):
    import paged_kv_cache_168_gb300 as pkv
    pkv.build_tables(s["qsl"], s["ctx"], s["slots"], s["positions"], s["tables"], s["free"], s["num_free"], s["left"], _desc(s), s["cached"], s["new"],
                     ring_blocks=s["case"]["ring"], dev_err=s["err"])
    return s["qsl"], s["ctx"], s["slots"], s["positions"], s["tables"], s["left"]


def _own_rope(s):
    import paged_kv_cache_168_gb300 as pkv
    pkv.rope_reshape_and_cache(s["q_out"], s["q"], s["pool"], _desc(s), s["key"], s["value"], s["slots"], s["positions"], s["cos_sin"], pair_axis=s["pair_axis"],
                               interleaved=s["case"]["pairs"], dev_err=s["err"])
    return s["q_out"], s["pool"]


def _own_extend(s):
    import paged_kv_cache_168_gb300 as pkv
    if s["ws"] is None:
        n = pkv.extend_workspace_bytes(_desc(s), s["ctx"].shape[0], s["q"].shape[0], s["q"].shape[1], s["max_q"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    pkv.extend(s["out"], s["q"], s["pool"], _desc(s), s["tables"], s["ctx"], s["qsl"], s["max_q"], s["scale"], s["ws"], window=s["case"]["window"],
               ring_blocks=s["ring"], dev_err=s["err"])
    return s["out"]


def _plain_tables(s):
    c = s["case"]
    bs, ring = c["bs"], c["ring"]
    old, new, tables, free = s["cached"].long(), s["new"].long(), s["tables"].long(), s["free"].long()
    ctx = old + new
    ends = torch.cumsum(new, 0)
    qsl = torch.cat([torch.zeros_like(ends[:1]), ends])
    have, need = (old + bs - 1) // bs, (ctx + bs - 1) // bs
    if ring:
        have, need = have.clamp(max=ring), need.clamp(max=ring)
    took = need - have
    first = torch.cumsum(took, 0) - took
    col = torch.arange(tables.shape[1], device=tables.device)[None, :]
    k = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    tables = torch.where(fresh, free[(s["num_free"].long() - 1 - k).clamp(0, free.shape[0] - 1)], tables)
    i = torch.arange(s["slots"].shape[0], device=tables.device)
    seq = torch.searchsorted(ends, i, right=True).clamp(max=old.shape[0] - 1)
    pos = old[seq] + i - qsl[seq]
    blk = pos // bs
    kept = i < ends[-1]
    positions = torch.where(kept, pos, 0)
    if ring:
        kept &= blk > (ctx[seq] - 1) // bs - ring
        blk = blk % ring
    slots = torch.where(kept, tables[seq, blk.clamp(0, tables.shape[1] - 1)] * bs + pos % bs, -1)
    i32 = torch.int32
    return qsl.to(i32), ctx.to(i32), slots, positions.to(i32), tables.to(i32), (s["num_free"] - took.sum()).to(i32)


def _chunk_index(bs, d, device):
    """Where element (part, token, dim) of a 16-bit chunk lies: groups of 8 tokens, K rows then V rows, 64-dim atoms, pieces at c xor r."""
    R = min(bs, 8)
    p, t, x = torch.arange(2, device=device)[:, None, None], torch.arange(bs, device=device)[None, :, None], torch.arange(d, device=device)[None, None, :]
    r = t % R
    return ((t // R * 2 + p) * (d // 64) + x // 64) * (R * 64) + r * 64 + ((x % 64 // 8) ^ r) * 8 + x % 8


def _code_index(bs, device):
    """Where code (part, token, dim) of an 8-bit chunk lies: 128-byte rows, pieces at c xor (t mod 8)."""
    p, t, x = torch.arange(2, device=device)[:, None, None], torch.arange(bs, device=device)[None, :, None], torch.arange(128, device=device)[None, None, :]
    return (p * bs + t) * 128 + ((x // 16) ^ (t % 8)) * 16 + x % 16


def _plain_rope(s):
    c = s["case"]
    bs, d, rot, hkv = c["bs"], c["d"], c["rot"], c["hkv"]
    dev = s["q"].device
    axis = torch.from_numpy(s["pair_axis"].astype(np.int64)).to(dev)
    pair = torch.arange(rot // 2, device=dev)
    at = s["positions"].long()[axis].t()                               # [T, pairs]
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, pair + rot // 2][:, None]

    def turned(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["pairs"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y1, y2 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y1, y2], -1).flatten(-2) if c["pairs"] else torch.cat([y1, y2], -1)
        return torch.cat([y, x[..., rot:]], -1)

    q, k, v = turned(s["q"]).to(s["q"].dtype), turned(s["key"]), s["value"].float()
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    blk, t = slot // bs, slot % bs
    kv = torch.stack([k[keep], v[keep]], 1)                            # [n, 2, hkv, d]
    h = torch.arange(hkv, device=dev)[None, None, :, None]
    b4 = blk[:, None, None, None]
    if not c["kv8"]:
        idx = _chunk_index(bs, d, dev).permute(1, 0, 2)[t][:, :, None, :]
        s["pool"][b4, h, idx] = kv.to(s["pool"].dtype)
        return q, s["pool"]
    amax = kv.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))
    code = (kv * inv).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    s["pool"][b4, h, _code_index(bs, dev).permute(1, 0, 2)[t][:, :, None, :]] = code
    sb = -(-4 * bs // 16) * 16
    part = torch.arange(2, device=dev)[None, :, None, None]
    s["pool"].view(torch.float32)[b4, h, (2 * bs * d + part * sb) // 4 + t[:, None, None, None]] = amax / 127
    return q, s["pool"]


def _plain_kv(s, ids):
    """K and V [.., 2, bs, d] in fp32 of the blocks `ids` [..]."""
    c = s["case"]
    bs, d = c["bs"], c["d"]
    got = s["pool"][ids]                                               # [.., hkv, chunk]
    if not c["kv8"]:
        return got[..., _chunk_index(bs, d, got.device)].float()
    codes = got[..., _code_index(bs, got.device)].view(torch.int8).float()
    sb = -(-4 * bs // 16) * 16
    scales = got[..., 2 * bs * d:].contiguous().view(torch.float32).unflatten(-1, (2, sb // 4))[..., :bs]
    return codes * scales[..., None]


def _plain_extend(s):
    c = s["case"]
    bs, d, hkv, ring, w = c["bs"], c["d"], c["hkv"], s["ring"], c["window"]
    dev, S = s["q"].device, s["ctx"].shape[0]
    G = c["hq"] // hkv
    ctx, qsl = s["ctx"].long(), s["qsl"].long()
    q_len = qsl[1:] - qsl[:-1]
    # logical blocks that any query may need, from the first held one on
    nb = -(-s["max_ctx"] // bs)
    base = torch.zeros_like(ctx)
    if ring:
        nb = min(nb, ring)
        base = ((ctx - 1) // bs - ring + 1).clamp(min=0)
    blk = base[:, None] + torch.arange(nb, device=dev)
    used = blk * bs < ctx[:, None]
    ids = torch.where(used, torch.gather(s["tables"].long(), 1, blk % ring if ring else blk.clamp(max=s["tables"].shape[1] - 1)), 0)
    kv = _plain_kv(s, ids)                                             # [S, nb, hkv, 2, bs, d]
    k = kv[:, :, :, 0].permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * bs, d)
    v = kv[:, :, :, 1].permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * bs, d)
    del kv
    j = torch.arange(s["max_q"], device=dev)[None, :]
    tok = (qsl[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][tok].float().unflatten(2, (hkv, G)).permute(0, 2, 1, 3, 4).reshape(S, hkv, -1, d)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])          # [S, hkv, max_q * G, nb * bs]
    pos = (ctx - q_len)[:, None] + j
    t = base[:, None] * bs + torch.arange(nb * bs, device=dev)
    see = t[:, None, :] <= pos[:, :, None]
    if w:
        see &= t[:, None, :] > pos[:, :, None] - w
    see = see[:, None, :, None, :].expand(S, 1, j.shape[1], G, t.shape[1]).reshape(S, 1, -1, t.shape[1])
    z.masked_fill_(~see, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).reshape(S, j.shape[1], hkv * G, d).to(s["q"].dtype)
    i = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(qsl[1:].contiguous(), i, right=True).clamp(max=S - 1)
    return o[seq, i - qsl[seq]]


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    return _exact_rope(s) if case["op"] == "rope" else _exact_extend(s)


def _exact_rope(s):
    """q as complex numbers turned by their angles; the 16-bit cache with every kept token's vectors in place."""
    c = s["case"]
    T, d, rot, bs, hkv = c["tokens"], c["d"], c["rot"], c["bs"], c["hkv"]
    n = rot // 2
    turn = torch.empty((T, n), dtype=torch.complex128, device=DEV)
    for i in range(n):
        a = s["positions"][int(s["pair_axis"][i])].double() * 10000.0 ** (-2 * i / rot)
        turn[:, i] = torch.polar(torch.ones_like(a), a)

    def go(x):
        y = x.double()
        first = torch.arange(n, device=DEV) * 2 if c["pairs"] else torch.arange(n, device=DEV)
        second = first + (1 if c["pairs"] else n)
        zc = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = zc.real, zc.imag
        return y

    q = go(s["q"])
    if c["kv8"]:
        return [q, None]  # codes are the fp32 values' roundings: whole numbers, not a 64-bit value
    pool = s["pool"].double()
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][keep]
    dims = torch.arange(d, device=DEV)
    R = min(bs, 8)
    for part, x in enumerate((go(s["key"]), s["value"].double())):
        for h in range(hkv):
            t = slot % bs
            row = (t // R * 2 + part) * (d * R) + (t % R) * 64
            off = row[:, None] + dims // 64 * (R * 64) + torch.bitwise_xor(dims // 8 % 8, (t % R)[:, None]) * 8 + dims % 8
            pool[(slot // bs)[:, None], h, off] = x[keep, h]
    return [q, pool]


def _exact_extend(s):
    """Sequence by sequence and kv head by kv head, from logical K and V."""
    c = s["case"]
    bs, d, hkv, ring, w, G = c["bs"], c["d"], c["hkv"], s["ring"], c["window"], c["hq"] // c["hkv"]
    qsl, ctxs = s["qsl"].tolist(), s["ctx"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    dims = torch.arange(d, device=DEV)
    for b, ctx in enumerate(ctxs):
        a, e = qsl[b], qsl[b + 1]
        if a == e:
            continue
        first = max(0, ((ctx - 1) // bs - ring + 1) * bs) if ring else 0
        if w:
            first = max(first, ctx - (e - a) - w + 1)
        t = torch.arange(first, ctx, device=DEV)
        blk = t // bs
        ids = s["tables"][b].long()[blk % ring if ring else blk]
        sl = t % bs
        pos = torch.arange(ctx - (e - a), ctx, device=DEV).repeat_interleave(G)
        bad = (t[None] > pos[:, None]) | ((t[None] <= pos[:, None] - w) if w else torch.zeros((), dtype=torch.bool, device=DEV))
        for h in range(hkv):
            kv = []
            for part in (0, 1):
                if c["kv8"]:
                    off = (part * bs + sl)[:, None] * 128 + torch.bitwise_xor(dims // 16, (sl % 8)[:, None]) * 16 + dims % 16
                    x = s["pool"][ids[:, None], h, off].view(torch.int8).double()
                    f = s["pool"].view(torch.float32)[ids, h, bs * d // 2 + part * (-(-bs // 4) * 4) + sl].double()
                    kv.append(x * f[:, None])
                else:
                    R = min(bs, 8)
                    off = ((sl // R * 2 + part) * (d * R) + sl % R * 64)[:, None] + dims // 64 * (R * 64) + torch.bitwise_xor(dims // 8 % 8, (sl % R)[:, None]) * 8 + dims % 8
                    kv.append(s["pool"][ids[:, None], h, off].double())
            z = s["q"][a:e, h * G:(h + 1) * G].double().reshape(-1, d) @ kv[0].T / math.sqrt(d)
            z[bad] = -math.inf
            o = torch.nan_to_num(torch.softmax(z, -1)) @ kv[1]
            out[a:e, h * G:(h + 1) * G] = o.view(e - a, G, d)
    return out
