"""Plain 64-bit (and, where bits are fixed, plain fp32) restatements of the paged-cache calls:
gdn_cache_tables row by row, gdn_cache_append token by token, attention request by request.
Nothing here uses the library."""
import numpy as np
import torch

F8 = torch.float8_e4m3fn
MIN_SCALE = np.float32(2.0 ** -64)


def e4m3_values():
    """Value of each of the 256 bytes: 1-4-3 bits, bias 7, subnormals, 0x7F / 0xFF NaN, no infinity."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


E4M3 = e4m3_values()
_MAG = E4M3[:127]  # 0 .. 448, ascending


def to_e4m3(x):
    """Bytes of the nearest e4m3 values (ties to the even byte) of fp32 numbers, +-448 beyond."""
    x = np.asarray(x, np.float32).astype(np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(_MAG, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _MAG[lo], _MAG[hi] - a
    b = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    b = np.where(np.isnan(x), 127, b)
    return (b | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def tables(lens_old, lens_new, table, ring, pool, bs, capacity):
    """The step's tables, row by row. Returns a dict of the outputs and whether rows were refused."""
    table, ring = table.copy(), ring.copy()
    N, (head, count) = ring.size, (int(pool[0]), int(pool[1]))
    B = len(lens_old)
    cap = table.shape[1] * bs
    n = lambda l: -(-l // bs)  # noqa: E731
    cu, slots, positions, lens = [0], [], [], []
    asked = taken = tail = 0
    bad = short = False
    for b in range(B):
        o, w = int(lens_old[b]), int(lens_new[b])
        if not (0 <= o <= cap and 0 <= w <= cap):
            bad, o, w = True, 0, 0
        need = max(0, n(w) - n(o))
        asked += need
        ok = need == 0 or asked <= count
        if need and ok:
            for j in range(need):
                table[b, n(o) + j] = ring[(head + asked - need + j) % N]
            taken = asked
        short |= not ok
        for t in range(max(0, w - o)):
            p = o + t
            positions.append(p)
            slots.append(int(table[b, p // bs]) * bs + p % bs if ok else -1)
        cu.append(cu[-1] + max(0, w - o))
        lens.append(w if ok else o)
    given = []
    for b in range(B):
        o, w = int(lens_old[b]), int(lens_new[b])
        if 0 <= o <= cap and 0 <= w <= cap:
            given += [int(table[b, j]) for j in range(n(w), n(o))]
    for g in given:
        ring[(head + count + tail) % N] = g
        tail += 1
    over = len(slots) > capacity
    pad = [-1] * max(0, capacity - len(slots))
    return {"table": table, "ring": ring, "pool": np.array([(head + taken) % N, count - taken + tail]),
            "cu": np.array(cu), "slots": np.array((slots + pad)[:capacity]),
            "positions": np.array((positions + pad)[:capacity]), "lens": np.array(lens),
            "bad": bad or over, "short": short}


def append(x, slots, cache, scale):
    """The writer on numpy arrays: x [T, H, d] fp32 (bf16 values), cache bytes [NB, H, bs, d], scale
    [NB, H] fp32. Runs token by token in fp32, as the definition has it."""
    cache, scale = cache.copy(), scale.copy()
    NB, H, bs, d = cache.shape
    t = 0
    while t < len(slots):
        s0 = int(slots[t])
        if s0 < 0 or s0 >= NB * bs:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and int(slots[t + n]) == s0 + n and (s0 + n) % bs:
            n += 1
        blk, off = s0 // bs, s0 % bs
        for h in range(H):
            v = x[t:t + n, h].astype(np.float32)
            fin = np.abs(v[np.isfinite(v)])
            a = np.float32(fin.max() if fin.size else 0.0)
            s = max(np.float32(a * np.float32(1.0 / 448.0)), MIN_SCALE)
            if off:
                s = max(s, scale[blk, h])
            r = np.float32(1.0) / s
            if off and s != scale[blk, h]:
                old = E4M3[cache[blk, h, :off]].astype(np.float32)
                cache[blk, h, :off] = to_e4m3((old * scale[blk, h]).astype(np.float32) * r)
            with np.errstate(invalid="ignore"):
                cache[blk, h, off:off + n] = to_e4m3(v * r)
            scale[blk, h] = s
        t += n
    return cache, scale


def attention(q, cu, kc, vc, ks, vs, table, lens, scale, p_bits, p_floor):
    """out [T, Hq, d] in 64 bits and an elementwise bound on a kernel's error, from what it rounds:
    a probability to `p_bits` bits and not below p_floor (relative to the row's largest), queries to
    2^-18 of their largest element, sums in fp32, the output to bf16. cu None: one token a request."""
    dev = q.device
    lut = torch.from_numpy(E4M3).to(dev)
    T, Hq, d = q.shape
    NB, H, bs, _ = kc.shape
    G = Hq // H
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    cu = list(range(len(lens) + 1)) if cu is None else [int(c) for c in cu]
    for b, n in enumerate(int(x) for x in lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or n <= 0:
            continue
        pages = table[b, : -(-n // bs)].long()
        good = (pages >= 0) & (pages < NB)
        seen = torch.repeat_interleave(good, bs)[:n]
        pages = pages.clamp(0, NB - 1)
        mask = torch.arange(n, device=dev)[None, :] <= (n - (hi - lo) + torch.arange(hi - lo, device=dev))[:, None]
        mask = mask & seen[None, :]
        any_key = mask.any(dim=1)
        for h in range(H):
            k = (lut[kc[pages, h].long()] * ks[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            v = (lut[vc[pages, h].long()] * vs[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            v = torch.where(seen[:, None], v, 0.0)
            k = torch.where(seen[:, None], k, 0.0)
            for m in range(h * G, (h + 1) * G):
                x = q[lo:hi, m].double()
                s = torch.where(mask, (x @ k.T) * scale, -torch.inf)
                top = s.amax(dim=1, keepdim=True)
                top = torch.where(torch.isinf(top), 0.0, top)
                p = torch.exp(s - top)
                z = p.sum(dim=1, keepdim=True)
                zz = torch.where(z > 0, z, 1.0)
                o = (p @ v) / zz
                out[lo:hi, m] = torch.where(any_key[:, None], o, 0.0)
                # a score is off by the query's rounding and by fp32 sums and exponents
                e = (2.0 ** -17 + d * 2.0 ** -23) * x.abs().amax(dim=1, keepdim=True) * k.abs().sum(dim=1).amax() * abs(scale)
                e = e + 2.0 ** -21 * (1 + torch.where(mask, s, 0.0).abs().amax(dim=1, keepdim=True))
                mag = (p @ v.abs()) / zz
                small = (torch.clamp(p, max=p_floor) @ torch.ones_like(v) * v.abs().amax()) / zz
                tol[lo:hi, m] = ((2.0 ** -p_bits + 2 * e + n * 2.0 ** -23) * mag + small + 2.0 ** -8 * o.abs()) * 1.01 + 1e-30
    return out, tol
