"""The 4-bit side of a hybrid model's attention step: rotary positions for q and k, the writer of the 4-bit paged cache
and its read-back, and the attention that reads that cache, for single tokens and for prompts. A "store" case is a write
and the read-back of what it wrote; every other case is one call.

Cache: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) in groups of 32 along the head, each group with a power of two
2^(byte - 127). k_cache [num_blocks, Hkv, block, d / 2] holds elements 2 i (low four bits) and 2 i + 1 of a token in a byte;
v_cache [num_blocks, Hkv, block / 2, d] holds an element of tokens 2 j (low four bits) and 2 j + 1; k_scale and v_scale
[num_blocks, Hkv, block, d / 32] are the groups' bytes.
"""
import math

import torch

own = False

DEV = "cuda"
E8 = torch.float8_e8m0fnu
BF16 = torch.bfloat16
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GROUP = 32
LEAST = -64              # the smallest exponent that is written


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 requests: heads of 256 with positions in their first quarter, up to 16,000 tokens in
        {"name": "rope decode 64", "op": "rope", "tokens": 64, "q_heads": 16, "kv_heads": 2, "dim": 256, "rot": 64,
         "interleaved": False, "scaling": "none", "factor": 1.0, "base": 1.0e7, "trained": 0, "max_pos": 16000},
        # a batch of prompts far into a long context, whole heads in pairs of neighbours, frequencies scaled by parts
        {"name": "rope prompts 31779", "op": "rope", "tokens": 31779, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": True, "scaling": "yarn", "factor": 16.0, "base": 1.0e6, "trained": 32768, "max_pos": 500000},
        # the cache write of a decode step: one token into partly filled blocks; read back as a check or a copy does
        {"name": "store decode 256", "op": "store", "batch": 256, "kv_heads": 2, "dim": 256, "block": 64, "max_new": 1,
         "max_len": 2048},
        # the cache write of a batch of prompts, odd lengths, some continuing a partly filled block
        {"name": "store prompts", "op": "store", "batch": 12, "kv_heads": 8, "dim": 128, "block": 32, "max_new": 4096,
         "max_len": 2048},
        # a long request's keys and values taken out of the cache, to move it or to work on it elsewhere
        {"name": "read 131071", "op": "read", "batch": 1, "kv_heads": 2, "dim": 256, "block": 128, "max_new": 131071,
         "max_len": 131071},
        # the smallest attention call: one request of a few thousand tokens, where latency counts
        {"name": "decode4 1 x 4097", "op": "decode", "batch": 1, "q_heads": 16, "kv_heads": 2, "dim": 256, "block": 64,
         "min_len": 4097, "max_len": 4097},
        # the ordinary serving batch, ragged, small pages, an odd number of heads to a group
        {"name": "decode4 64 ragged", "op": "decode", "batch": 64, "q_heads": 28, "kv_heads": 4, "dim": 128, "block": 16,
         "min_len": 1, "max_len": 8192},
        # few rows over a long axis: two requests with a long context
        {"name": "decode4 2 x 131071", "op": "decode", "batch": 2, "q_heads": 16, "kv_heads": 2, "dim": 256, "block": 128,
         "min_len": 131071, "max_len": 131071},
        # the largest decode batch: 256 requests around 8,000 tokens
        {"name": "decode4 256 x 8192", "op": "decode", "batch": 256, "q_heads": 16, "kv_heads": 2, "dim": 256, "block": 64,
         "min_len": 7000, "max_len": 8192},
        # one whole prompt at the repository's prefill length
        {"name": "prefill4 4096", "op": "prefill", "batch": 1, "q_heads": 16, "kv_heads": 2, "dim": 256, "block": 64,
         "min_new": 4096, "max_new": 4096, "min_old": 0, "max_old": 0},
        # eight ragged prompts, some with a cached prefix
        {"name": "prefill4 varlen 8", "op": "prefill", "batch": 8, "q_heads": 16, "kv_heads": 4, "dim": 64, "block": 16,
         "min_new": 1, "max_new": 4096, "min_old": 0, "max_old": 700},
        # a piece of a long prompt: few rows over a long axis
        {"name": "prefill4 300 at 60000", "op": "prefill", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "block": 64,
         "min_new": 300, "max_new": 300, "min_old": 60000, "max_old": 60000},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "read", "decode", "decode", "prefill", "prefill"])
    block, dim, kv = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while group * kv > 32:
        group = rng.choice([1, 2, 3, 4])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, dim // 2 - 2])
        scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
        return {"op": op, "tokens": _log(rng, 1, min(32768, 150_000_000 // (dim * (group + 1) * kv))), "q_heads": group * kv,
                "kv_heads": kv, "dim": dim, "rot": rot, "interleaved": rng.random() < 0.5, "scaling": scaling,
                "factor": 1.0 if scaling == "none" else float(rng.choice([2, 4, 8, 32])),
                "base": float(rng.choice([10000, 500000, 10000000])), "trained": rng.choice([2048, 8192, 32768]),
                "max_pos": _log(rng, 64, 1000000)}
    if op == "store":
        batch = _log(rng, 1, 256)
        return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "block": block,
                "max_new": _log(rng, 1, max(1, 24576 // batch)), "max_len": _log(rng, 16, 4096)}
    if op == "read":
        batch = _log(rng, 1, 64)
        top = _log(rng, 1, max(1, 67_000_000 // (batch * kv * dim)))
        return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "block": block, "max_new": top, "max_len": top}
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
    """New tokens and tokens before them, of each request. The sizes of a case do not go by the seed, so that its work is
    one number; the seed makes the values and the pages' order."""
    g, B = _gen(11, 1), case["batch"]
    if case["op"] == "decode":
        return torch.ones(B, dtype=torch.int64), _between(g, case["min_len"], case["max_len"], B) - 1
    if case["op"] == "prefill":
        new = _between(g, case["min_new"], case["max_new"], B)
        return new, _between(g, case["min_old"], case["max_old"], B)
    if case["op"] == "read":     # from the request's start
        return _between(g, (case["max_new"] + 1) // 2 if B > 1 else case["max_new"], case["max_new"], B), torch.zeros(B, dtype=torch.int64)
    return _between(g, 1, case["max_new"], B), _between(g, 0, case["max_len"], B)


def _cdiv(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------------------- inputs

def _freqs(case):
    """The angle of each pair per position, in 64 bits, and the factor of the rotated values."""
    r, base, f = case["rot"], case["base"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64)
    if case["scaling"] == "ntk" and r > 2:
        base = base * f ** (r / (r - 2))
    w = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] != "yarn":
        return w, 1.0
    # pairs that turn 32 times or more over the trained length keep their frequency, those that turn once or less are
    # divided by the factor, the ones between go from one to the other along their index
    at = [r * math.log(case["trained"] / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
    mix = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return w / f * mix + w * (1.0 - mix), 0.1 * math.log(f) + 1.0


def _quantise(x):
    """Codes (0 .. 15) and group bytes of fp32 values whose last axis is the head: 2^e the least power of two with all of
    the group at most 7 * 2^e, codes rounded to nearest, ties to the even code."""
    x = x.unflatten(-1, (-1, GROUP))
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=-1)
    m, e = torch.frexp(top)                       # top = m 2^e, m in [0.5, 1): at most 7 * 2^(e - 3) up to m = 7/8
    e = torch.where(m <= 0.875, e - 3, e - 2)
    e = torch.where(top > 0, e, LEAST).clamp(min=LEAST)
    y = torch.ldexp(x, -e[..., None])
    a = y.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a > edge) if i % 2 == 0 else (a >= edge)     # a tie goes to the even code
    code |= torch.signbit(y).to(torch.uint8) << 3
    byte = torch.where(torch.isnan(x).any(dim=-1), 255, e + 127)
    return code.flatten(-2), byte.to(torch.uint8)


def _cache(case, nblocks, seed):
    """A cache that holds values: per channel and per token of other sizes, as keys and values are."""
    g = torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))
    H, bs, d = case["kv_heads"], case["block"], case["dim"]
    kc = torch.empty(nblocks, H, bs, d // 2, dtype=torch.uint8, device=DEV)
    vc = torch.empty(nblocks, H, bs // 2, d, dtype=torch.uint8, device=DEV)
    ks, vs = (torch.empty(nblocks, H, bs, d // GROUP, dtype=torch.uint8, device=DEV) for _ in "kv")
    for which in "kv":
        size = torch.exp(0.5 * torch.randn(H, 1, d, device=DEV, generator=g))
        step = max(1, (1 << 26) // (H * bs * d))
        for a in range(0, nblocks, step):
            n = min(step, nblocks - a)
            x = torch.randn(n, H, bs, d, device=DEV, generator=g).mul_(size)
            x.mul_(torch.exp(0.3 * torch.randn(n, H, bs, 1, device=DEV, generator=g)))
            code, byte = _quantise(x)
            if which == "k":
                kc[a:a + n], ks[a:a + n] = code[..., 0::2] | code[..., 1::2] << 4, byte
            else:
                vc[a:a + n], vs[a:a + n] = code[:, :, 0::2] | code[:, :, 1::2] << 4, byte
    return {"kc": kc, "vc": vc, "ks": ks.view(E8), "vs": vs.view(E8)}


def _pages(lens, block, width, spare, seed):
    """A shuffled block table [B, width] for the given lengths, -1 past them, and the pool's size."""
    n = _cdiv(lens, block)
    total = int(n.sum()) + spare
    perm = torch.randperm(total, generator=_gen(seed, 4))
    first = torch.cumsum(n, 0) - n
    j = torch.arange(width)[None, :]
    used = j < n[:, None]
    return torch.where(used, perm[(first[:, None] + j).clamp(max=total - 1)], -1).to(torch.int32), total


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device=DEV).manual_seed((int(seed) + 1) % (1 << 62))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op == "rope":
        T, Hq, H, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        qkv = torch.randn(T, Hq + 2 * H, d, device=DEV, generator=g).to(BF16)    # q, k and v are slices of one projection
        # requests at places of their own, their tokens in order
        starts = torch.randint(0, case["max_pos"], (_cdiv(T, 512),), generator=_gen(seed, 6))
        pos = (starts[:, None] + torch.arange(512)).reshape(-1)[:T] if T > 512 else torch.randint(0, case["max_pos"], (T,), generator=_gen(seed, 6))
        freqs, factor = _freqs(case)
        s = {"op": op, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "pos": pos.to(torch.int32).to(DEV), "freqs": freqs.to(DEV),
             "factor": factor, "rot": case["rot"], "interleaved": case["interleaved"],
             "q_out": torch.empty(T, Hq, d, dtype=BF16, device=DEV), "k_out": torch.empty(T, H, d, dtype=BF16, device=DEV)}
        if own:     # the table of a model's frequencies is made once
            import gated_deltanet_linear_gdn_gb300 as gdn
            s["rope"] = gdn.RopeTable(case["rot"], base=case["base"], scaling=case["scaling"], factor=case["factor"],
                                      trained_len=case["trained"], device=DEV)
        return s
    new, old = _lens(case)
    lens, bs, H, d = new + old, case["block"], case["kv_heads"], case["dim"]
    table, total = _pages(lens, bs, int(_cdiv(lens, bs).max()), 3, seed)
    s = {"op": op, "err": err, **_cache(case, total, seed)}
    T = int(new.sum())
    if op in ("store", "read"):
        row = torch.repeat_interleave(torch.arange(case["batch"]), new)
        pos = old[row] + torch.arange(T) - (torch.cumsum(new, 0) - new)[row]
        s["slots"] = (table[row, pos // bs].long() * bs + pos % bs).to(torch.int32).to(DEV)
        s["k_back"], s["v_back"] = torch.empty(2, T, H, d, dtype=BF16, device=DEV)
        if op == "store":
            kv = torch.randn(T, 2, H, d, device=DEV, generator=g) * torch.exp(0.5 * torch.randn(H, d, device=DEV, generator=g))
            kv = kv.to(BF16)    # k and v are slices of one projection: a token stride of 2 H d
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
        return s
    Hq = case["q_heads"]
    q = (1.5 * torch.randn(T, Hq, d, device=DEV, generator=g)).to(BF16)
    s.update(q=q, table=table.to(DEV), lens=lens.to(torch.int32).to(DEV), out=torch.empty_like(q),
             cu=torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)]).to(torch.int32).to(DEV),
             most_new=int(new.max()), heads=(Hq, H, d), blocks=int(_cdiv(lens, bs).sum()))
    # a server keeps one scratch buffer for its attention calls
    s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _plain_rope(s):
    angle = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = (f(angle).float()[:, None, :] * s["factor"] for f in (torch.cos, torch.sin))
    r, out = s["rot"], {}
    for name in "qk":
        x = s[name].float()
        y = x.clone()
        a, b = (slice(0, r, 2), slice(1, r, 2)) if s["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        s[name + "_out"].copy_(y)
        out[name] = s[name + "_out"]
    return out


def _values(codes, scales):
    """fp32 values of codes [..., d] with group bytes [..., d / 32]."""
    lut = torch.tensor(MAGNITUDES + [-m for m in MAGNITUDES], device=codes.device)
    return (lut[codes.int()].unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _plain_store(s):
    slots = s["slots"].long()
    bs = s["kc"].shape[2]
    blk, off = slots // bs, slots % bs
    code, byte = _quantise(s["k"].float())
    s["kc"][blk, :, off] = code[..., 0::2] | code[..., 1::2] << 4
    s["ks"].view(torch.uint8)[blk, :, off] = byte
    code, byte = _quantise(s["v"].float())
    for odd in (0, 1):      # two tokens share a byte: one after the other
        at = torch.nonzero(off % 2 == odd)[:, 0]
        was = s["vc"][blk[at], :, off[at] // 2]
        s["vc"][blk[at], :, off[at] // 2] = (was & 15 | code[at] << 4) if odd else (was & 240 | code[at])
    s["vs"].view(torch.uint8)[blk, :, off] = byte
    return {**_plain_read(s), "k_scale": s["ks"], "v_scale": s["vs"]}


def _plain_read(s):
    slots = s["slots"].long()
    bs = s["kc"].shape[2]
    blk, off = slots // bs, slots % bs
    k = s["kc"][blk, :, off]
    v = s["vc"][blk, :, off // 2] >> (off % 2 * 4).to(torch.uint8)[:, None, None] & 15
    ks, vs = (s[n].view(torch.uint8)[blk, :, off].view(E8) for n in ("ks", "vs"))
    s["k_back"].copy_(_values(torch.stack([k & 15, k >> 4], dim=-1).flatten(-2), ks))
    s["v_back"].copy_(_values(v, vs))
    return {"k": s["k_back"], "v": s["v_back"]}


def _plain_attention(s):
    """softmax(scale q k^T) v, all requests at once, padded to the longest."""
    Hq, H, d = s["heads"]
    q, table, lens, cu, Q = s["q"], s["table"].long(), s["lens"].long(), s["cu"].long(), s["most_new"]
    B, bs = lens.numel(), s["kc"].shape[2]
    L = table.shape[1] * bs
    pick = table.clamp(min=0)

    def heads_first(x):     # [B, W, H, bs, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, d)

    def keys():
        c = s["kc"][pick]
        return heads_first(_values(torch.stack([c & 15, c >> 4], dim=-1).flatten(-2), s["ks"].view(torch.uint8)[pick].view(E8)))

    def values():
        c = s["vc"][pick]
        return heads_first(_values(torch.stack([c & 15, c >> 4], dim=4).flatten(3, 4), s["vs"].view(torch.uint8)[pick].view(E8)))

    i = torch.arange(Q, device=q.device)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                        # [B, Q]
    qq = q[at].float().reshape(B, Q, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * Q, d)
    sc = torch.matmul(qq, keys().transpose(2, 3)).mul_(d ** -0.5).reshape(B, H, Hq // H, Q, L)
    seen = torch.arange(L, device=q.device) <= (lens - n)[:, None, None] + i[:, None]      # [B, Q, L]
    seen &= torch.arange(L, device=q.device) < lens[:, None, None]
    sc.masked_fill_(~seen[:, None, None], -float("inf"))
    sc.sub_(sc.amax(dim=-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = sc.sum(dim=-1, keepdim=True)
    o = torch.matmul(sc.reshape(B, H, Hq // H * Q, L), values()).reshape(B, H, Hq // H, Q, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, d).to(BF16)
    return {"out": o[i[None, :] < n[:, None]]}


# ------------------------------------------------------------------------------------------ run

def run(state):
    s, op = state, state["op"]
    if not own:
        return {"rope": _plain_rope, "store": _plain_store, "read": _plain_read}.get(op, _plain_attention)(s)
    import gated_deltanet_linear_gdn_gb300 as gdn
    if op == "rope":
        gdn.gdn_rope(s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], s["rope"], interleaved=s["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cache = s["kc"], s["vc"], s["ks"], s["vs"]
    if op in ("store", "read"):
        if op == "store":
            gdn.gdn_cache4_append(s["k"], s["v"], s["slots"], *cache, err=s["err"])
        gdn.gdn_cache4_read(*cache, s["slots"], s["k_back"], s["v_back"], err=s["err"])
        back = {"k": s["k_back"], "v": s["v_back"]}
        return {**back, "k_scale": s["ks"], "v_scale": s["vs"]} if op == "store" else back
    if op == "decode":
        gdn.gdn_attn4_decode(s["q"], *cache, s["table"], s["lens"], s["out"], s["workspace"], err=s["err"])
    else:
        gdn.gdn_attn4_prefill(s["q"], s["cu"], *cache, s["table"], s["lens"], s["out"], s["workspace"],
                              held_blocks=s["blocks"], err=s["err"])
    return {"out": s["out"]}


# ----------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "rope":
        T, heads, d, r = case["tokens"], case["q_heads"] + case["kv_heads"], case["dim"], case["rot"]
        return {"bytes": T * (heads * d * 4 + 4) + 4 * r, "flops": T * heads * r * 3}
    new, old = _lens(case)
    H, d, T = case["kv_heads"], case["dim"], int(new.sum())
    token = 2 * H * (d // 2 + d // GROUP)            # a token's bytes in the cache
    if case["op"] == "read":
        return {"bytes": T * (4 + token + 4 * H * d), "flops": 0}
    if case["op"] == "store":                         # bf16 in, the cache, bf16 out
        return {"bytes": T * (4 + token + 8 * H * d), "flops": 0}
    lens, Hq = new + old, case["q_heads"]
    pairs = int((new * old + new * (new + 1) // 2).sum())
    return {"bytes": int(lens.sum()) * token + 4 * int(_cdiv(lens, case["block"]).sum()) + T * Hq * d * 4,
            "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------------------------------- exact

def _e2m1(code):
    """Values of codes by their bits: two of exponent (bias 1), one of fraction."""
    e, m = (code >> 1 & 3).double(), (code & 1).double()
    v = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)
    return torch.where((code & 8) > 0, -v, v)


def _token(s, which, slot):
    """64-bit values [H, n, d] of the tokens in the given slots."""
    bs = s["kc"].shape[2]
    blk, off = slot // bs, slot % bs
    if which == "k":
        byte = s["kc"][blk, :, off]
        code = torch.empty(*byte.shape[:2], 2 * byte.shape[2], dtype=torch.int64, device=byte.device)
        code[..., 0::2], code[..., 1::2] = byte.long() % 16, byte.long() // 16
    else:
        code = s["vc"][blk, :, off // 2].long() // (16 ** (off % 2))[:, None, None] % 16
    e = s[which + "s"].view(torch.uint8)[blk, :, off].double() - 127
    return (_e2m1(code) * torch.exp2(e).repeat_interleave(GROUP, dim=2)).transpose(0, 1)


def _nearest(x):
    """64-bit numbers [T, H, d] as the cache holds them, and their groups' scales."""
    x = x.double().reshape(*x.shape[:2], -1, GROUP)
    top = x.abs().amax(dim=-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top / 7)).clamp(min=LEAST))
    scale = torch.where(top > 7 * scale, 2 * scale, torch.where((top <= 3.5 * scale) & (scale > 2.0 ** LEAST), scale / 2, scale))
    y = x / scale
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)     # the spacing of the values around y
    return (torch.round(y / unit) * unit).clamp(-6.0, 6.0).mul(scale).flatten(2), scale[..., 0]


def exact(case, seed):
    """Each operator from its definition in 64 bits: angles and rotations, values and scales, attention request by request
    and head by head."""
    s = prepare(case, seed)
    if case["op"] == "rope":
        r, w = case["rot"], s["freqs"].cpu()
        turn = torch.polar(torch.ones_like(w)[None, :], s["pos"].cpu().double()[:, None] * w).to(DEV)[:, None, :] * s["factor"]
        out = {}
        for name in "qk":
            x = s[name].double()
            pair = x[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            out[name] = torch.cat([(y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2), x[..., r:]], dim=-1)
        return out
    if case["op"] in ("store", "read"):
        out, slot, bs = {}, s["slots"].long(), case["block"]
        for which in "kv":
            if case["op"] == "read":
                out[which] = _token(s, which, slot).transpose(0, 1)
            else:
                out[which], scale = _nearest(s[which])
                pool = s[which + "s"].double()
                pool[slot // bs, :, slot % bs] = scale
                out[which + "_scale"] = pool
        return out
    Hq, H, d = s["heads"]
    G, bs = Hq // H, case["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    for b, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        slot = s["table"][b, at // bs].long() * bs + at % bs
        k, v = _token(s, "k", slot), _token(s, "v", slot)
        a, e = cu[b], cu[b + 1]
        hidden = at[None, :] > (n - (e - a) + torch.arange(e - a, device=DEV))[:, None]
        for m in range(Hq):
            x = s["q"][a:e, m].double() @ k[m // G].T / math.sqrt(d)
            x[hidden] = -math.inf
            out[a:e, m] = torch.softmax(x, dim=-1) @ v[m // G]
    return {"out": out}
