"""The attention side of a hybrid model's step, as a server calls it next to the GDN layers: the
block tables of the step, the 8-bit paged cache's writer, and the attention that reads the cache,
for single tokens and for prompts. Each case is one call.

Cache: k_cache, v_cache [num_blocks, Hkv, block, d] in e4m3 with k_scale, v_scale [num_blocks, Hkv]
in fp32; an element stands for byte * scale.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
MIN_SCALE = 2.0 ** -64   # the writer's smallest scale: a block of zeros keeps a positive one
INV_MAX = 1.0 / 448.0    # 1 / the largest e4m3 value


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 requests: a token each, a new block for the few that cross into one
        {"name": "tables decode 64", "op": "tables", "batch": 64, "block": 64, "long": 0.0, "drop": 0.0,
         "max_len": 8192, "max_new": 1},
        # a busy mixed step: decode rows, prompts of up to 512 tokens, finished requests giving blocks back
        {"name": "tables mixed 1024", "op": "tables", "batch": 1024, "block": 16, "long": 0.2, "drop": 0.1,
         "max_len": 16384, "max_new": 512},
        # the cache write of a decode step: one token into partly filled blocks
        {"name": "append decode 256", "op": "append", "batch": 256, "kv_heads": 2, "dim": 256, "block": 64,
         "max_new": 1, "max_len": 2048},
        # the cache write of a batch of prompts, odd lengths, some continuing a partly filled block
        {"name": "append prompts", "op": "append", "batch": 12, "kv_heads": 8, "dim": 128, "block": 32,
         "max_new": 4096, "max_len": 2048},
        # the smallest call: one request of a few thousand tokens, where latency counts
        {"name": "decode 1 x 4097", "op": "decode", "batch": 1, "q_heads": 16, "kv_heads": 2, "dim": 256,
         "block": 64, "min_len": 4097, "max_len": 4097},
        # an odd batch of short and middling requests, heads in groups of seven, small pages
        {"name": "decode 33 ragged", "op": "decode", "batch": 33, "q_heads": 28, "kv_heads": 4, "dim": 64,
         "block": 16, "min_len": 1, "max_len": 3000},
        # the ordinary serving batch, ragged
        {"name": "decode 64 ragged", "op": "decode", "batch": 64, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "block": 32, "min_len": 1, "max_len": 8192},
        # few rows over a long axis: two requests with a long context
        {"name": "decode 2 x 131071", "op": "decode", "batch": 2, "q_heads": 16, "kv_heads": 2, "dim": 256,
         "block": 128, "min_len": 131071, "max_len": 131071},
        # the largest decode batch: 256 requests around 8,000 tokens
        {"name": "decode 256 x 8192", "op": "decode", "batch": 256, "q_heads": 16, "kv_heads": 2, "dim": 256,
         "block": 64, "min_len": 7000, "max_len": 8192},
        # one whole prompt at the repository's prefill length
        {"name": "prefill 4096", "op": "prefill", "batch": 1, "q_heads": 16, "kv_heads": 2, "dim": 256,
         "block": 64, "min_new": 4096, "max_new": 4096, "min_old": 0, "max_old": 0},
        # eight ragged prompts, some with a cached prefix
        {"name": "prefill varlen 8", "op": "prefill", "batch": 8, "q_heads": 16, "kv_heads": 4, "dim": 128,
         "block": 16, "min_new": 1, "max_new": 4096, "min_old": 0, "max_old": 700},
        # a piece of a long prompt: few rows over a long axis
        {"name": "prefill 300 at 60000", "op": "prefill", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "block": 64, "min_new": 300, "max_new": 300, "min_old": 60000, "max_old": 60000},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "prefill", "prefill"])
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        return {"op": op, "batch": _log(rng, 1, 1024), "block": block, "long": round(rng.uniform(0, 0.5), 3),
                "drop": round(rng.uniform(0, 0.3), 3), "max_len": _log(rng, 64, 16384), "max_new": _log(rng, 1, 512)}
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        batch = _log(rng, 1, 256)
        return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "block": block,
                "max_new": _log(rng, 1, max(1, 32768 // batch)), "max_len": _log(rng, 16, 4096)}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while group * kv > 32:
        group = rng.choice([1, 2, 3, 4])
    if op == "decode":
        batch = _log(rng, 1, 256)
        top = _log(rng, 16, max(16, min(131072, 800_000_000 // (batch * kv * dim))))
        return {"op": op, "batch": batch, "q_heads": group * kv, "kv_heads": kv, "dim": dim, "block": block,
                "min_len": max(1, top // rng.choice([1, 2, 1000])), "max_len": top}
    batch = rng.choice([1, 1, 2, 3, 5, 8])
    new = _log(rng, 1, 4096 if batch <= 2 else 2048)
    old = _log(rng, 1, 20000 if batch * new <= 1024 else 1500) - 1
    while 4 * dim * group * kv * batch * new * (old + new / 2) > 2.2e11:    # no more than the largest listed one
        new = new * 2 // 3
    return {"op": op, "batch": batch, "q_heads": group * kv, "kv_heads": kv, "dim": dim, "block": block,
            "min_new": max(1, new // rng.choice([1, 3, 100])), "max_new": new, "min_old": old // 2, "max_old": old}


# ---------------------------------------------------------------------------------------- sizes

def _gen(seed, k):
    return torch.Generator().manual_seed((int(seed) * 1000003 + k) % (1 << 62))


def _between(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _lens(case):
    """Lengths of a decode or prefill case: (new tokens, cached before). The sizes of a case do not go
    by the seed, so that its work is one number; the seed makes the values and the pages' order."""
    g, B = _gen(7, 1), case["batch"]
    if case["op"] == "decode":
        return torch.ones(B, dtype=torch.int64), _between(g, case["min_len"], case["max_len"], B) - 1
    new = _between(g, case["min_new"], case["max_new"], B)
    return new, _between(g, case["min_old"], case["max_old"], B)


def _append_lens(case):
    g, B = _gen(7, 2), case["batch"]
    return _between(g, 1, case["max_new"], B), _between(g, 0, case["max_len"], B)


def _table_lens(case):
    g, B = _gen(7, 3), case["batch"]
    old = _between(g, 1, case["max_len"], B)
    new = old + 1
    kind = torch.rand(B, generator=g)
    grown = _between(g, 1, case["max_new"], B)
    new = torch.where(kind < case["long"], old + grown, new)
    # prompts that begin in this step
    fresh = torch.rand(B, generator=g) < 0.5
    begins = (kind < case["long"]) & fresh
    old, new = torch.where(begins, 0, old), torch.where(begins, grown, new)
    new = torch.where(kind > 1 - case["drop"], 0, new)   # finished: all blocks go back
    return old, new


def _cdiv(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------------------- inputs

def _cache(case, nblocks, seed):
    """A cache that holds values: per channel and per block of other sizes, as keys and values are."""
    g = torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))
    H, bs, d = case["kv_heads"], case["block"], case["dim"]
    out = []
    for _ in range(2):
        size = torch.exp(0.5 * torch.randn(H, 1, d, device=DEV, generator=g))
        each = torch.exp(0.3 * torch.randn(nblocks, H, 1, 1, device=DEV, generator=g))
        x = torch.randn(nblocks, H, bs, d, device=DEV, generator=g, dtype=torch.float32)
        x = x.mul_(size).mul_(each)
        s = (x.abs().amax(dim=(2, 3)) * INV_MAX).clamp_(min=MIN_SCALE)
        x = x.mul_((1.0 / s)[:, :, None, None]).clamp_(-448.0, 448.0)
        out += [x.to(F8), s]
        del x
    return out[0], out[2], out[1], out[3]


def _pages(lens, block, width, spare, seed):
    """A shuffled block table [B, width] for the given lengths, -1 past them, and the pool's size."""
    n = _cdiv(lens, block)
    total = int(n.sum()) + spare
    perm = torch.randperm(total, generator=_gen(seed, 4))
    first = torch.cumsum(n, 0) - n
    j = torch.arange(width)[None, :]
    used = j < n[:, None]
    table = torch.where(used, perm[(first[:, None] + j).clamp(max=total - 1)], -1).to(torch.int32)
    return table, total, perm[int(n.sum()):]


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device=DEV).manual_seed((int(seed) + 1) % (1 << 62))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op == "tables":
        old, new = _table_lens(case)
        bs, B = case["block"], case["batch"]
        width = int(_cdiv(torch.maximum(old, new), bs).max()) + 1
        need = int((_cdiv(new, bs) - _cdiv(old, bs)).clamp(min=0).sum())
        table, total, free = _pages(old, bs, width, need + 7, seed)
        head = int(torch.randint(0, total, (1,), generator=_gen(seed, 5)))
        ring = torch.full((total,), -1, dtype=torch.int32)
        ring[(head + torch.arange(free.numel())) % total] = free.to(torch.int32)
        T = int((new - old).clamp(min=0).sum()) + 5       # capacity: a little padding at the end
        i32 = dict(dtype=torch.int32, device=DEV)
        return {"op": op, "block": bs, "old": old.to(**i32), "new": new.to(**i32), "table": table.to(DEV),
                "ring": ring.to(DEV), "pool": torch.tensor([head, free.numel()], **i32),
                "pool_out": torch.zeros(2, **i32), "cu": torch.zeros(B + 1, **i32),
                "slots": torch.zeros(T, **i32), "positions": torch.zeros(T, **i32),
                "lens": torch.zeros(B, **i32), "err": err}
    if op == "append":
        new, old = _append_lens(case)
        bs, H, d = case["block"], case["kv_heads"], case["dim"]
        table, total, _ = _pages(old + new, bs, int(_cdiv(old + new, bs).max()), 3, seed)
        row = torch.repeat_interleave(torch.arange(case["batch"]), new)
        pos = old[row] + torch.arange(row.numel()) - (torch.cumsum(new, 0) - new)[row]
        slots = table[row, pos // bs].long() * bs + pos % bs
        kc, vc, ks, vs = _cache(case, total, seed)
        T = row.numel()
        kv = torch.randn(T, 2, H, d, device=DEV, generator=g) * torch.exp(0.5 * torch.randn(H, d, device=DEV, generator=g))
        kv = kv.to(torch.bfloat16)    # k and v are slices of one projection: a token stride of 2 H d
        return {"op": op, "k": kv[:, 0], "v": kv[:, 1], "slots": slots.to(torch.int32).to(DEV), "kc": kc, "vc": vc,
                "ks": ks, "vs": vs, "err": err}
    new, old = _lens(case)
    lens = new + old
    bs, d, Hq = case["block"], case["dim"], case["q_heads"]
    table, total, _ = _pages(lens, bs, int(_cdiv(lens, bs).max()), 3, seed)
    kc, vc, ks, vs = _cache(case, total, seed)
    T = int(new.sum())
    q = (1.5 * torch.randn(T, Hq, d, device=DEV, generator=g)).to(torch.bfloat16)
    s = {"op": op, "q": q, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table.to(DEV),
         "lens": lens.to(torch.int32).to(DEV), "out": torch.empty_like(q), "err": err,
         "cu": torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)]).to(torch.int32).to(DEV),
         "most_new": int(new.max()), "heads": (Hq, case["kv_heads"], d)}
    # a server keeps one scratch buffer for its attention calls
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _plain_tables(s):
    bs, old, new, table, ring = s["block"], s["old"].long(), s["new"].long(), s["table"], s["ring"]
    N, T = ring.numel(), s["slots"].numel()
    head, count = s["pool"][0].long(), s["pool"][1].long()
    n_old, n_new = (old + bs - 1) // bs, (new + bs - 1) // bs
    need, give = (n_new - n_old).clamp(min=0), (n_old - n_new).clamp(min=0)
    upto, back = torch.cumsum(need, 0), torch.cumsum(give, 0)
    refused = (need > 0) & (upto > count)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    # blocks given back go to the ring's tail; blocks taken come from its head
    gives = (j >= n_new[:, None]) & (j < n_old[:, None])
    at = (head + count + (back - give)[:, None] + j - n_new[:, None]) % N
    ring_out = torch.cat([ring, ring[:1]])
    ring_out[torch.where(gives, at, N)] = table
    takes = (j >= n_old[:, None]) & (j < n_new[:, None]) & ~refused[:, None]
    at = (head + (upto - need)[:, None] + j - n_old[:, None]) % N
    table = torch.where(takes, ring[at], table)
    taken = torch.where(refused, 0, need).sum()
    q = (new - old).clamp(min=0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=q.device), torch.cumsum(q, 0)])
    t = torch.arange(T, device=q.device)
    row = torch.searchsorted(cu[1:], t, right=True)
    real = row < old.numel()
    row = row.clamp(max=old.numel() - 1)
    pos = old[row] + t - cu[row]
    slot = table[row, (pos // bs).clamp(0, table.shape[1] - 1)].long() * bs + pos % bs
    slot = torch.where(real & ~refused[row], slot, -1)
    i = torch.int32
    return {"table": table, "ring": ring_out[:-1],
            "pool": torch.stack([(head + taken) % N, count - taken + back[-1]]).to(i), "cu": cu.to(i),
            "slots": slot.to(i), "positions": torch.where(real, pos, -1).to(i),
            "lens": torch.where(refused, old, new).to(i)}


def _plain_write(x, slots, cache, scale):
    NB, H, bs, d = cache.shape
    x = x.float()
    live = slots >= 0
    blk, off = torch.where(live, slots // bs, NB), slots % bs          # skipped tokens go to a block past the end
    mag = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=2)      # [T, H]
    top = torch.zeros(NB + 1, H, device=x.device).scatter_reduce(0, blk[:, None].expand(-1, H), mag, "amax")[:NB]
    first = torch.full((NB + 1,), bs, device=x.device, dtype=off.dtype).scatter_reduce(0, blk, off, "amin")[:NB]
    touched, partly = first < bs, (first < bs) & (first > 0)
    s = torch.maximum(top * INV_MAX, torch.where(partly[:, None], scale, 0.0)).clamp(min=MIN_SCALE)
    s = torch.where(touched[:, None], s, scale)
    r = 1.0 / s
    # tokens that were there: written anew where their scale grew
    at, raw = torch.nonzero(partly)[:, 0], cache.view(torch.uint8)
    old = raw[at].view(F8).float()
    again = ((old * scale[at][:, :, None, None]) * r[at][:, :, None, None]).clamp(-448.0, 448.0).to(F8).float()
    stays = (torch.arange(bs, device=x.device)[None, :] >= first[at][:, None])[:, None, :, None] | (s[at] == scale[at])[:, :, None, None]
    raw[at] = torch.where(stays, old, again).to(F8).view(torch.uint8)
    byte = (x * r[blk.clamp(max=NB - 1)][:, :, None]).clamp(-448.0, 448.0).to(F8)
    raw[blk[live], :, off[live]] = byte.view(torch.uint8)[live]
    scale.copy_(s)


def _plain_append(s):
    slots = s["slots"].long()
    _plain_write(s["k"], slots, s["kc"], s["ks"])
    _plain_write(s["v"], slots, s["vc"], s["vs"])
    return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _plain_attention(s):
    """softmax(scale q k^T) v, all requests at once, padded to the longest."""
    Hq, H, d = s["heads"]
    q, table, lens, cu, Q = s["q"], s["table"].long(), s["lens"].long(), s["cu"].long(), s["most_new"]
    B, bs = lens.numel(), s["kc"].shape[2]
    L = table.shape[1] * bs
    pick = table.clamp(min=0)

    def values(cache, scale):
        x = cache.view(torch.uint8)[pick].view(F8).float() * scale[pick][..., None, None]    # [B, W, H, bs, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, d)

    i = torch.arange(Q, device=q.device)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                        # [B, Q]
    qq = q[at].float().reshape(B, Q, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * Q, d)
    sc = torch.matmul(qq, values(s["kc"], s["ks"]).transpose(2, 3)).mul_(d ** -0.5).reshape(B, H, Hq // H, Q, L)
    seen = torch.arange(L, device=q.device) <= (lens - n)[:, None, None] + i[:, None]      # [B, Q, L]
    seen &= torch.arange(L, device=q.device) < lens[:, None, None]
    sc.masked_fill_(~seen[:, None, None], -float("inf"))
    sc.sub_(sc.amax(dim=-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = sc.sum(dim=-1, keepdim=True)
    o = torch.matmul(sc.reshape(B, H, Hq // H * Q, L), values(s["vc"], s["vs"])).reshape(B, H, Hq // H, Q, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, d).to(torch.bfloat16)
    return {"out": o[i[None, :] < n[:, None]]}


# ------------------------------------------------------------------------------------------ run

def run(state):
    s = state
    if not own:
        return {"tables": _plain_tables, "append": _plain_append}.get(s["op"], _plain_attention)(s)
    import gated_deltanet_linear_gdn_gb300 as gdn
    if s["op"] == "tables":
        gdn.gdn_cache_tables(s["old"], s["new"], s["table"], s["ring"], s["pool"], s["pool_out"], s["cu"], s["slots"],
                             s["positions"], s["lens"], s["block"], err=s["err"])
        return {"table": s["table"], "ring": s["ring"], "pool": s["pool_out"], "cu": s["cu"], "slots": s["slots"],
                "positions": s["positions"], "lens": s["lens"]}
    if s["op"] == "append":
        gdn.gdn_cache_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"], err=s["err"])
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if s["op"] == "decode":
        gdn.gdn_attn_decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["out"],
                            s["workspace"], err=s["err"])
    else:
        gdn.gdn_attn_prefill(s["q"], s["cu"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["out"],
                             s["workspace"], err=s["err"])
    return {"out": s["out"]}


# ----------------------------------------------------------------------------------------- work

def work(case):
    op, bs = case["op"], case["block"]
    if op == "tables":
        old, new = _table_lens(case)
        blocks = int((_cdiv(new, bs) - _cdiv(old, bs)).abs().sum())
        T = int((new - old).clamp(min=0).sum()) + 5
        return {"bytes": 4 * (4 * case["batch"] + 2 * blocks + 2 * T), "flops": 0}
    if op == "append":
        new, old = _append_lens(case)
        row = case["kv_heads"] * case["dim"]
        touched = int((_cdiv(old + new, bs) - old // bs).sum())
        return {"bytes": int(new.sum()) * (4 + 2 * row * 3) + touched * case["kv_heads"] * 2 * 4, "flops": 0}
    new, old = _lens(case)
    lens, d, Hq, H = new + old, case["dim"], case["q_heads"], case["kv_heads"]
    pairs = int((new * old + new * (new + 1) // 2).sum())
    blocks = int(_cdiv(lens, bs).sum())
    return {"bytes": int(lens.sum()) * H * d * 2 + blocks * (4 + 8 * H) + int(new.sum()) * Hq * d * 4,
            "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------------------------------- exact

def _to_e4m3(x):
    """The nearest e4m3 value (ties to even) of 64-bit numbers, at most 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_write(x, slots, cache, scale):
    """The cache after the write, block by block: its values before the scale, and the scales."""
    bs, out, s = cache.shape[2], cache.double(), scale.double()
    by = {}
    for t, slot in enumerate(slots.tolist()):
        by.setdefault(slot // bs, []).append((slot % bs, t))
    for blk, put in by.items():
        off, tok = (torch.tensor(v, device=x.device) for v in zip(*put))
        new, first = x[tok].double(), int(off.min())
        top = new.abs().amax(dim=(0, 2)) / 448
        if first:
            top = torch.maximum(top, s[blk])
            grown = top > s[blk]
            kept = out[blk, grown, :first] * s[blk, grown, None, None] / top[grown, None, None]
            out[blk, grown, :first] = _to_e4m3(kept)
        s[blk] = top
        out[blk, :, off] = _to_e4m3(new / top[:, None]).transpose(0, 1)
    return out, s


def exact(case, seed):
    """Attention and the cache's values from their definitions in 64 bits, request by request and head
    by head, block by block. The tables are whole numbers."""
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        (k, ks), (v, vs) = (_exact_write(s[a], s["slots"], s[a + "c"], s[a + "s"]) for a in "kv")
        return {"k_cache": k, "v_cache": v, "k_scale": ks, "v_scale": vs}
    Hq, H, d = s["heads"]
    G, bs = Hq // H, case["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    for b, n in enumerate(lens):
        pages = s["table"][b, : _cdiv(n, bs)].long()
        a, e = cu[b], cu[b + 1]
        hidden = torch.arange(n, device=DEV)[None, :] > (n - (e - a) + torch.arange(e - a, device=DEV))[:, None]
        for h in range(H):
            k = (s["kc"].view(torch.uint8)[pages, h].view(F8).double() * s["ks"][pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            v = (s["vc"].view(torch.uint8)[pages, h].view(F8).double() * s["vs"][pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            for m in range(h * G, (h + 1) * G):
                x = s["q"][a:e, m].double() @ k.T / math.sqrt(d)
                x[hidden] = -math.inf
                out[a:e, m] = torch.softmax(x, dim=-1) @ v
    return {"out": out}
