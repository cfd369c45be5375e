"""Plain restatements of the 4-bit cache's calls and of rotary positions: the format bit by bit, the writer token by token,
attention request by request in 64 bits. Nothing here uses the library."""
import math

import numpy as np
import torch

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAG, -MAG])
LEAST = -64


def nearest_code(y):
    """Codes of 64-bit numbers: the nearest value, ties to the even code, +-6 beyond; the sign is kept."""
    a = np.minimum(np.abs(y), 6.0)
    hi = np.clip(np.searchsorted(MAG, a), 1, 7)
    lo = hi - 1
    dl, dh = a - MAG[lo], MAG[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def quantise(x):
    """Codes and bytes of the groups of one token's head, x [d] (bf16 values); None for the codes of a group with NaN."""
    codes, scales = [], []
    for g in x.reshape(-1, 32).astype(np.float64):
        if np.isnan(g).any():
            codes.append(None)
            scales.append(255)
            continue
        top = np.abs(g[np.isfinite(g)]).max(initial=0.0)
        e = LEAST
        while top > 7.0 * 2.0 ** e:
            e += 1
        codes.append(nearest_code(g / 2.0 ** e))
        scales.append(e + 127)
    return codes, scales


def append(k, v, slots, kc, vc, ks, vs):
    """The writer on numpy arrays, token by token. The codes of a group with NaN are left as they were."""
    kc, vc, ks, vs = kc.copy(), vc.copy(), ks.copy(), vs.copy()
    NB, H, bs, _ = kc.shape
    for t, s in enumerate(slots):
        if s < 0 or s >= NB * bs:
            continue
        blk, off = s // bs, s % bs
        for h in range(H):
            for i, (code, byte) in enumerate(zip(*quantise(k[t, h]))):
                ks[blk, h, off, i] = byte
                if code is not None:
                    kc[blk, h, off, 16 * i:16 * i + 16] = code[0::2] | code[1::2] << 4
            for i, (code, byte) in enumerate(zip(*quantise(v[t, h]))):
                vs[blk, h, off, i] = byte
                if code is not None:
                    at = vc[blk, h, off // 2, 32 * i:32 * i + 32]
                    vc[blk, h, off // 2, 32 * i:32 * i + 32] = (at & 15) | code << 4 if off % 2 else (at & 240) | code
    return kc, vc, ks, vs


def unpack(kc, vc, ks, vs):
    """64-bit values [NB, H, bs, d] of a whole cache (torch, any device)."""
    lut = torch.from_numpy(VALUES).to(kc.device)
    k = lut[torch.stack([kc & 15, kc >> 4], dim=-1).flatten(-2).long()]
    v = lut[torch.stack([vc & 15, vc >> 4], dim=3).flatten(2, 3).long()]

    def scale(b):
        e = torch.exp2(b.double() - 127)
        return torch.where(b == 255, torch.nan, e).repeat_interleave(32, dim=3)

    return k * scale(ks), v * scale(vs)


def attention(q, cu, k, v, table, lens, scale, p_bits, p_floor, k_off=0.0, v_off=0.0, v_exp=0):
    """out [T, Hq, d] in 64 bits over unpacked values k, v [NB, H, bs, d], and an elementwise bound on a kernel's error: a
    probability rounded to `p_bits` bits (half a step is 2^-p_bits of it) and not below p_floor of the row's largest
    probability x value, fp32 sums of the scores and of the output, the output's rounding to bf16 (2^-8); k_off and v_off:
    what a key or value may be off by, relative to the largest that the request holds; v_exp: the largest |log2| of V's scales,
    which an exponent is added to and the maximum taken from in fp32 (three roundings of half a step, 2^-24 of it each)."""
    dev = q.device
    T, Hq, d = q.shape
    NB, H, bs, _ = k.shape
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
        mask = (torch.arange(n, device=dev)[None, :] <= (n - (hi - lo) + torch.arange(hi - lo, device=dev))[:, None]) & seen[None, :]
        any_key = mask.any(dim=1)
        for h in range(H):
            kk = torch.where(seen[:, None], k[pages, h].reshape(-1, d)[:n], 0.0)
            vv = torch.where(seen[:, None], v[pages, h].reshape(-1, d)[:n], 0.0)
            for m in range(h * G, (h + 1) * G):
                x = q[lo:hi, m].double()
                s = torch.where(mask, (x @ kk.T) * scale, -torch.inf)
                top = s.amax(dim=1, keepdim=True)
                top = torch.where(torch.isinf(top), 0.0, top)
                p = torch.exp(s - top)
                z = p.sum(dim=1, keepdim=True)
                zz = torch.where(z > 0, z, 1.0)
                o = torch.where(mask, p, 0.0) @ vv / zz
                out[lo:hi, m] = torch.where(any_key[:, None], o, 0.0)
                # a score: products of d terms in fp32 (and queries to 2^-17 of their largest), the exponent
                big = x.abs().amax(dim=1, keepdim=True) * kk.abs().sum(dim=1).amax() * abs(scale)
                e = (2.0 ** -17 + d * 2.0 ** -23 + k_off * d) * big
                e = e + 2.0 ** -21 * (1 + torch.where(mask, s, 0.0).abs().amax(dim=1, keepdim=True))
                e = e + 3 * 2.0 ** -24 * v_exp
                mag = (p @ vv.abs()) / zz
                most = (p[:, :, None] * vv.abs().amax(dim=1)[None, :, None]).amax(dim=1) if p.numel() < 1 << 22 else vv.abs().amax()
                small = n * p_floor * most / zz + v_off * vv.abs().amax()
                tol[lo:hi, m] = ((2.0 ** -p_bits + 2 * e + n * 2.0 ** -23) * mag + small + 2.0 ** -8 * o.abs()) * 1.01 + 1e-30
    return out, tol


def rope(x, positions, freqs, factor, rot, interleaved):
    """64-bit rotation of x [T, h, d], and a bound on a kernel's error: sines, cosines and products in fp32 from an angle
    that is off by 2^-30 of a turn, one rounding to bf16 (2^-8)."""
    x = x.double()
    a = positions.double()[:, None] * torch.as_tensor(freqs, dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(a)[:, None, :] * factor, torch.sin(a)[:, None, :] * factor
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    size = (x[..., i].abs() + x[..., j].abs()) * factor
    off = 2 * math.pi * 2.0 ** -30 + 2.0 ** -21   # the angle; sines, their factor, two products and a sum: a few 2^-24
    tol[..., i] = size * off + y[..., i].abs() * 2.0 ** -8
    tol[..., j] = size * off + y[..., j].abs() * 2.0 ** -8
    return y, tol * 1.01 + 1e-30
