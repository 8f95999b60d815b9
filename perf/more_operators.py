"""Cases and plain forms of the operators of layers with normed heads and shaped scores.

norm     norms of q and k for each head, rotary positions and the cache write in one pass
extend   attention of a chunk of new tokens per sequence over the paged cache, with scores capped by a tanh or
         lowered by distance, and a span of positions of its own for each query (documents, prefixes)
decode   the same for one token per sequence

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
    N, E, D = "norm", "extend", "decode"
    return [
        # the new token of 256 decoding requests, grouped heads
        dict(name="norm_decode", op=N, tokens=256, hq=32, hkv=8, d=128, rot=128, bs=16, dtype="bf16", offset=False, pairs=False, far=8192),
        # a batch of whole prompts
        dict(name="norm_prompts", op=N, tokens=32768, hq=32, hkv=8, d=128, rot=128, bs=16, dtype="bf16", offset=True, pairs=False, far=131072),
        # ragged prompts, small heads, an odd number of heads a group, half of each head rotated, neighbouring pairs
        dict(name="norm_small_heads", op=N, tokens=5001, hq=15, hkv=5, d=64, rot=32, bs=8, dtype="f16", offset=False, pairs=True, far=4096),
        # the smallest call: a handful of new tokens over short contexts, where latency counts
        dict(name="extend_tiny", op=E, seqs=4, q_lo=1, q_hi=5, pre_lo=0, pre_hi=95, hq=4, hkv=4, d=64, bs=16, dtype="f16", kv8=False, window=0, cap=50.0,
             slopes=False, doc=0, prefix=0, holes=False),
        # chunked prefill under a cap: 512-token chunks over cached prefixes
        dict(name="extend_capped", op=E, seqs=32, q_lo=512, q_hi=512, pre_lo=512, pre_hi=3584, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=False, window=0,
             cap=50.0, slopes=False, doc=0, prefix=0, holes=False),
        # whole prompts whose scores fall with distance, a slope for each of as many query as kv heads
        dict(name="extend_slopes", op=E, seqs=16, q_lo=2048, q_hi=2048, pre_lo=0, pre_hi=0, hq=32, hkv=32, d=128, bs=16, dtype="f16", kv8=False, window=0,
             cap=0.0, slopes=True, doc=0, prefix=0, holes=False),
        # documents packed into long rows, each with a prefix that sees itself whole; padding tokens that see nothing
        dict(name="extend_documents", op=E, seqs=2, q_lo=8192, q_hi=8192, pre_lo=0, pre_hi=0, hq=32, hkv=8, d=128, bs=32, dtype="bf16", kv8=False, window=0,
             cap=0.0, slopes=False, doc=2000, prefix=300, holes=True),
        # ragged chunks over an 8-bit cache, capped, a sliding window
        dict(name="extend_int8", op=E, seqs=32, q_lo=1, q_hi=700, pre_lo=1, pre_hi=3500, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=True, window=1500,
             cap=30.0, slopes=False, doc=0, prefix=0, holes=False),
        # checking four drafted tokens a request against long contexts, capped
        dict(name="extend_verify", op=E, seqs=8, q_lo=4, q_hi=4, pre_lo=32764, pre_hi=131068, hq=64, hkv=8, d=128, bs=32, dtype="bf16", kv8=False, window=0,
             cap=50.0, slopes=False, doc=0, prefix=0, holes=False),
        # single tokens, a slope for each head
        dict(name="decode_slopes", op=D, seqs=64, q_lo=1, q_hi=1, pre_lo=511, pre_hi=4095, hq=32, hkv=32, d=128, bs=16, dtype="f16", kv8=False, window=0,
             cap=0.0, slopes=True, doc=0, prefix=0, holes=False),
        # single tokens of many requests, capped, grouped heads
        dict(name="decode_capped", op=D, seqs=256, q_lo=1, q_hi=1, pre_lo=0, pre_hi=3000, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv8=False, window=0,
             cap=50.0, slopes=False, doc=0, prefix=0, holes=False),
        # few requests with long contexts in an 8-bit cache, capped
        dict(name="decode_int8", op=D, seqs=8, q_lo=1, q_hi=1, pre_lo=32767, pre_hi=131071, hq=64, hkv=8, d=128, bs=16, dtype="bf16", kv8=True, window=0,
             cap=30.0, slopes=False, doc=0, prefix=0, holes=False),
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
        if w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1] and _plain_cost(c) <= 4.5e9:
            return c


def _plain_cost(c):
    # scores of the plain form's padded rectangle
    return 0 if c["op"] == "norm" else c["seqs"] * c["hq"] * c["q_hi"] * (c["pre_hi"] + c["q_hi"])


def _draw(rng):
    op = rng.choice(["norm", "extend", "extend", "decode"])
    if op == "norm":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 32])
        return dict(op=op, tokens=_log(rng, 1, 32768), hq=hkv * rng.choice([1, 3, 4, 5, 8]), hkv=hkv, d=d, rot=rng.choice([d, d // 2]),
                    bs=rng.choice([1, 2, 4, 8, 16, 32]), dtype=rng.choice(["f16", "bf16"]), offset=rng.random() < 0.5, pairs=rng.random() < 0.5,
                    far=_log(rng, 1024, 131072))
    d = rng.choice([64, 128, 128])
    kv8 = d == 128 and rng.random() < 0.4
    hkv = rng.choice([1, 2, 4, 8, 32])
    q_hi = 1 if op == "decode" else _log(rng, 1, 2048)
    pre_hi = _log(rng, 1, 131068) if q_hi < 9 else _log(rng, 1, 9000)
    shape = rng.choice(["cap", "cap", "slopes", "both", "spans"])
    return dict(op=op, seqs=_log(rng, 1, 256 if op == "decode" else 64), q_lo=1 if op == "decode" else rng.randint(0 if q_hi > 1 else 1, q_hi), q_hi=q_hi,
                pre_lo=rng.randint(0, pre_hi), pre_hi=pre_hi, hq=hkv * rng.choice([1, 2, 4, 5, 8, 16]), hkv=hkv, d=d, bs=rng.choice([1, 4, 8, 16, 16, 32]),
                dtype=rng.choice(["f16", "bf16"]), kv8=kv8, window=rng.choice([0, 0, rng.randint(1, 2000)]),
                cap=rng.choice([5.0, 20.0, 30.0, 50.0, 100.0]) if shape in ("cap", "both") or (shape == "spans" and rng.random() < 0.5) else 0.0,
                slopes=shape in ("slopes", "both"), doc=_log(rng, 20, 4000) if shape == "spans" else 0,
                prefix=_log(rng, 1, 600) if shape == "spans" and op == "extend" and rng.random() < 0.6 else 0,
                holes=shape == "spans" and rng.random() < 0.5)


# ------------------------------------------------------------------ lengths and spans (on the host)

def _lens(case, seed):
    """Cached and new lengths of a case's requests, and which request of the case each is: a seed has an order of its own."""
    g = np.random.default_rng(7)
    S = case["seqs"]
    new, old = g.integers(case["q_lo"], case["q_hi"] + 1, S), g.integers(case["pre_lo"], case["pre_hi"] + 1, S)
    if new.sum() == 0:
        new[-1] = max(1, case["q_hi"])
    order = np.random.default_rng(seed & 0xFFFFFFFF).permutation(S)
    return old[order].astype(np.int64), new[order].astype(np.int64), order


def _spans(case, old, new, who):
    """First and last position that each query's span allows; None where the case has no spans."""
    if not case["doc"]:
        return None
    first, last = [], []
    for o, n, i in zip(old.tolist(), new.tolist(), who.tolist()):
        g = np.random.default_rng([11, i])
        # documents of a tenth of `doc` to `doc` tokens, each with a prefix of up to `prefix` tokens
        starts = np.concatenate([[0], np.cumsum(g.integers(max(1, case["doc"] // 10), case["doc"] + 1, (o + n) // max(1, case["doc"] // 10) + 1))])
        heads = g.integers(0, case["prefix"] + 1, len(starts))
        p = np.arange(o, o + n)
        k = np.searchsorted(starts, p, side="right") - 1
        ends = np.concatenate([starts[1:], [1 << 30]])
        a = starts[k]
        b = np.maximum(p, np.minimum(a + heads[k], ends[k]) - 1)
        if case["holes"]:
            a = np.where(g.random(n) < 0.02, b + 1, a)
        first.append(a)
        last.append(b)
    return np.concatenate(first).astype(np.int64), np.concatenate(last).astype(np.int64)


def _attended(case, old, new, spans):
    """Positions [lo, hi] of every query, request after request."""
    pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)])
    ctx = np.repeat(old + new, new)
    lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros_like(pos)
    if spans is None:
        return lo, pos
    return np.maximum(lo, spans[0]), np.minimum(ctx - 1, spans[1] if case["prefix"] else np.minimum(pos, spans[1]))


def work(case):
    if case["op"] == "norm":
        T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        return {"bytes": T * (4 * hq * d + 8 * hkv * d + 4 + 8), "flops": T * (hq + hkv) * (4 * d + 3 * case["rot"])}
    old, new, who = _lens(case, 0)
    lo, hi = _attended(case, old, new, _spans(case, old, new, who))
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    read = 0                                                         # cached tokens that some query attends
    at = np.concatenate([[0], np.cumsum(new)])
    for o, n, a, e in zip(old, new, at[:-1], at[1:]):
        mark = np.zeros(o + n + 1, np.int64)
        some = hi[a:e] >= lo[a:e]
        np.add.at(mark, lo[a:e][some], 1)
        np.add.at(mark, hi[a:e][some] + 1, -1)
        read += int((np.cumsum(mark) > 0).sum())
    kv = hkv * (2 * d + 8) if case["kv8"] else 4 * hkv * d
    T = int(new.sum())
    spans = 4 * T * ((case["doc"] > 0) + (case["prefix"] > 0))
    return {"bytes": 4 * T * hq * d + read * kv + 4 * (read // case["bs"] + 2 * case["seqs"]) + spans + (4 * hq if case["slopes"] else 0),
            "flops": float(4 * d * hq * int(np.maximum(0, hi - lo + 1).sum()))}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g, size=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(size).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _pool(case, nb, g):
    """Cache memory of nb blocks that holds normal values (16-bit), or codes and scales (8-bit)."""
    hkv, bs, d = case["hkv"], case["bs"], case["d"]
    if not case.get("kv8"):
        return torch.cat([_normal((min(4096, nb - i), hkv, 2 * bs * d), DTYPES[case["dtype"]], g) for i in range(0, nb, 4096)])
    sb = -(-4 * bs // 16) * 16
    pool = torch.zeros((nb, hkv, 2 * bs * d + 2 * sb), dtype=torch.uint8, device=DEV)
    for i in range(0, nb, 4096):
        n = min(4096, nb - i)
        x = torch.randn((n, hkv, 2 * bs * d), generator=g, device=DEV).mul_(127 / 3.2).round_().clamp_(-127, 127)
        pool[i:i + n, :, :2 * bs * d] = x.to(torch.int8).view(torch.uint8)
        s = (torch.rand((n, hkv, 2, sb // 4), generator=g, device=DEV) * 1.6 + 2.0) / 127
        pool[i:i + n, :, 2 * bs * d:] = s.view(n, hkv, -1).view(torch.uint8)
    return pool


def prepare(case, seed):
    return _prepare_norm(case, _gen(seed)) if case["op"] == "norm" else _prepare_attention(case, seed, _gen(seed))


def _prepare_norm(case, g):
    T, hq, hkv, d, rot, bs = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot", "bs"))
    dt, far = DTYPES[case["dtype"]], case["far"]
    nb = int(1.1 * T) // bs + 2
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    ang = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * inv
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:T].contiguous()
    slots[torch.rand(T, generator=g, device=DEV) < 0.02] = -1        # padding, and tokens that the cache holds already
    # vectors of very different lengths, as projections leave them
    size = lambda h: torch.exp(torch.randn((T, h, 1), generator=g, device=DEV))
    q = (_normal((T, hq, d), torch.float32, g) * size(hq)).to(dt)
    key = (_normal((T, hkv, d), torch.float32, g) * size(hkv)).to(dt)
    base = 0.0 if case["offset"] else 1.0
    weight = lambda: (_normal((d,), torch.float32, g, 0.2) + base).to(dt)
    return dict(case=case, q=q, q_out=torch.empty_like(q), key=key, value=_normal((T, hkv, d), dt, g), pool=_pool(case, nb, g), num_blocks=nb, slots=slots,
                positions=torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32), cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
                q_weight=weight(), k_weight=weight(), eps=1e-6, offset=1.0 if case["offset"] else 0.0, err=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_attention(case, seed, g):
    old, new, who = _lens(case, seed)
    S, hq, d, bs = case["seqs"], case["hq"], case["d"], case["bs"]
    ctx = old + new
    nblk = -(-ctx // bs)
    width = int(max(nblk.max(), 1))
    nb = int(1.05 * nblk.sum()) + 2
    h = torch.from_numpy(nblk).to(DEV)
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(h, 0) - h)[:, None] + col
    tables = torch.where(col < h[:, None], perm[at.clamp(max=nb - 1)], torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous()
    T = int(new.sum())
    # scores of a few units up to tens where they are capped
    q = _normal((T, hq, d), DTYPES[case["dtype"]], g, 4.0 if case["cap"] else 1.0)
    slopes = torch.from_numpy(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)).float().to(DEV) if case["slopes"] else None
    spans = _spans(case, old, new, who)
    return dict(case=case, q=q, out=torch.empty_like(q), pool=_pool(case, nb, g), num_blocks=nb, tables=tables, ctx=_i32(ctx),
                qsl=_i32(np.concatenate([[0], np.cumsum(new)])), max_q=int(new.max()), max_ctx=int(ctx.max()), scale=1 / math.sqrt(d), slopes=slopes,
                first=None if spans is None else _i32(spans[0]), last=_i32(spans[1]) if spans is not None and case["prefix"] else None,
                err=torch.zeros(1, dtype=torch.int32, device=DEV), ws=None)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own_norm(s) if op == "norm" else _own_extend(s) if op == "extend" else _own_decode(s)
    return _plain_norm(s) if op == "norm" else _plain_attention(s)


def _desc(s):
    """The cache's geometry, which a user's program keeps beside its pool."""
    if "desc" not in s:
        import paged_kv_cache_168_gb300 as pkv
        c = s["case"]
        s["desc"] = pkv.CacheDesc(s["num_blocks"], c["bs"], c["hkv"], c["d"], DTYPES[c["dtype"]], kv_int8=c.get("kv8", False))
    return s["desc"]


def _own_norm(s):
    import paged_kv_cache_168_gb300 as pkv
    pkv.norm_rope_reshape_and_cache(s["q_out"], s["q"], s["pool"], _desc(s), s["key"], s["value"], s["slots"], s["positions"], s["cos_sin"], s["q_weight"],
                                    s["k_weight"], s["eps"], weight_offset=s["offset"], interleaved=s["case"]["pairs"], dev_err=s["err"])
    return s["q_out"], s["pool"]


def _own_extend(s):
    import paged_kv_cache_168_gb300 as pkv
    if s["ws"] is None:
        n = pkv.extend_scored_workspace_bytes(_desc(s), s["ctx"].shape[0], s["q"].shape[0], s["q"].shape[1], s["max_q"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    pkv.extend_scored(s["out"], s["q"], s["pool"], _desc(s), s["tables"], s["ctx"], s["qsl"], s["max_q"], s["scale"], s["ws"], softcap=s["case"]["cap"],
                      slopes=s["slopes"], first_pos=s["first"], last_pos=s["last"], window=s["case"]["window"], dev_err=s["err"])
    return s["out"]


def _own_decode(s):
    import paged_kv_cache_168_gb300 as pkv
    if s["ws"] is None:
        n = pkv.decode_scored_workspace_bytes(_desc(s), s["ctx"].shape[0], s["q"].shape[1], s["max_ctx"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    pkv.decode_scored(s["out"], s["q"], s["pool"], _desc(s), s["tables"], s["ctx"], s["max_ctx"], s["scale"], s["ws"], softcap=s["case"]["cap"],
                      slopes=s["slopes"], first_pos=s["first"], window=s["case"]["window"], dev_err=s["err"])
    return s["out"]


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


def _plain_norm(s):
    c = s["case"]
    bs, d, rot, hkv = c["bs"], c["d"], c["rot"], c["hkv"]
    row = s["cos_sin"][s["positions"].long()][:, None]                 # [T, 1, rot]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]

    def turned(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * (weight.float() + s["offset"])
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["pairs"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y1, y2 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y1, y2], -1).flatten(-2) if c["pairs"] else torch.cat([y1, y2], -1)
        return torch.cat([y, x[..., rot:]], -1)

    q, k, v = turned(s["q"], s["q_weight"]).to(s["q"].dtype), turned(s["key"], s["k_weight"]), s["value"].float()
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    kv = torch.stack([k[keep], v[keep]], 1)                            # [n, 2, hkv, d]
    h = torch.arange(hkv, device=q.device)[None, None, :, None]
    idx = _chunk_index(bs, d, q.device).permute(1, 0, 2)[slot % bs][:, :, None, :]
    s["pool"][(slot // bs)[:, None, None, None], h, idx] = kv.to(s["pool"].dtype)
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


def _plain_attention(s):
    c = s["case"]
    bs, d, hkv, w = c["bs"], c["d"], c["hkv"], c["window"]
    dev, S = s["q"].device, s["ctx"].shape[0]
    G = c["hq"] // hkv
    ctx, qsl = s["ctx"].long(), s["qsl"].long()
    q_len = qsl[1:] - qsl[:-1]
    nb = -(-s["max_ctx"] // bs)
    blk = torch.arange(nb, device=dev)[None].expand(S, nb)
    ids = torch.where(blk * bs < ctx[:, None], s["tables"].long()[:, :nb], 0)
    kv = _plain_kv(s, ids)                                             # [S, nb, hkv, 2, bs, d]
    k = kv[:, :, :, 0].permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * bs, d)
    v = kv[:, :, :, 1].permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * bs, d)
    del kv
    j = torch.arange(s["max_q"], device=dev)[None, :]
    tok = (qsl[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][tok].float().unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, d)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])          # [S, hkv, G * max_q, nb * bs]
    del k
    if c["cap"]:
        z.div_(c["cap"]).tanh_().mul_(c["cap"])
    z = z.view(S, hkv, G, s["max_q"], nb * bs)
    pos = (ctx - q_len)[:, None] + j                                   # [S, max_q]
    t = torch.arange(nb * bs, device=dev)
    if s["slopes"] is not None:
        far = (pos[:, :, None] - t).abs().float()                      # [S, max_q, nb * bs]
        z.addcmul_(far[:, None, None], s["slopes"].view(1, hkv, G, 1, 1), value=-1)
    last = pos if s["last"] is None else s["last"].long()[tok]
    see = (t <= last[:, :, None]) & (t < ctx[:, None, None])
    if s["first"] is not None:
        see &= t >= s["first"].long()[tok][:, :, None]
    if w:
        see &= t > pos[:, :, None] - w
    z.masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hkv, -1, nb * bs), v).view(S, hkv, G, s["max_q"], d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, s["max_q"], hkv * G, d).to(s["q"].dtype)
    i = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(qsl[1:].contiguous(), i, right=True).clamp(max=S - 1)
    return o[seq, i - qsl[seq]]


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_attention(s)


def _exact_norm(s):
    """Vectors over their root mean square, as complex numbers turned by their angles; the cache with every kept token's vectors in place."""
    c = s["case"]
    T, d, rot, bs, hkv = c["tokens"], c["d"], c["rot"], c["bs"], c["hkv"]
    n = rot // 2
    turn = torch.empty((T, n), dtype=torch.complex128, device=DEV)
    for i in range(n):
        a = s["positions"].double() * 10000.0 ** (-2 * i / rot)
        turn[:, i] = torch.polar(torch.ones_like(a), a)
    first = torch.arange(n, device=DEV) * (2 if c["pairs"] else 1)
    second = first + (1 if c["pairs"] else n)

    def go(x, weight):
        y = x.double()
        y = y / (y.square().sum(-1, keepdim=True) / d + s["eps"]).sqrt() * (s["offset"] + weight.double())
        zc = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = zc.real, zc.imag
        return y

    pool = s["pool"].double()
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][keep]
    dims = torch.arange(d, device=DEV)
    R = min(bs, 8)
    for part, x in enumerate((go(s["key"], s["k_weight"]), s["value"].double())):
        for h in range(hkv):
            t = slot % bs
            row = (t // R * 2 + part) * (d * R) + (t % R) * 64
            off = row[:, None] + dims // 64 * (R * 64) + torch.bitwise_xor(dims // 8 % 8, (t % R)[:, None]) * 8 + dims % 8
            pool[(slot // bs)[:, None], h, off] = x[keep, h]
    return [go(s["q"], s["q_weight"]), pool]


def _exact_attention(s):
    """Sequence by sequence and kv head by kv head, from logical K and V, a thousand queries at a time."""
    c = s["case"]
    bs, d, hkv, G = c["bs"], c["d"], c["hkv"], c["hq"] // c["hkv"]
    qsl, ctxs = s["qsl"].tolist(), s["ctx"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    dims = torch.arange(d, device=DEV)
    for b, ctx in enumerate(ctxs):
        a0, e0 = qsl[b], qsl[b + 1]
        if a0 == e0:
            continue
        t = torch.arange(ctx, device=DEV)
        ids, sl = s["tables"][b].long()[t // bs], t % bs
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
            for a in range(a0, e0, 1024):
                e = min(e0, a + 1024)
                pos = torch.arange(ctx - (e0 - a), ctx - (e0 - e), device=DEV)
                z = torch.einsum("ngd,td->ngt", s["q"][a:e, h * G:(h + 1) * G].double(), kv[0]) / math.sqrt(d)
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][h * G:(h + 1) * G].double()[:, None] * (pos[:, None, None] - t).abs()
                bad = t > (pos if s["last"] is None else s["last"][a:e])[:, None]
                if s["first"] is not None:
                    bad = bad | (t < s["first"][a:e, None])
                if c["window"]:
                    bad = bad | (t <= pos[:, None] - c["window"])
                z.masked_fill_(bad[:, None], -math.inf)
                out[a:e, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.nan_to_num(torch.softmax(z, -1)), kv[1])
    return out
