"""The 4-bit writer and read-back where a CTA has several tokens at a time and takes them in several rounds, a thread two tokens
of values: narrow heads, and enough tokens for either call's rounds. The bytes are those of calls short enough for one round."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

from test_gpu_cache4 import cache, i32, same_values
import _cache4_oracle as co

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def in_rounds(H, d):
    """Tokens that are more than 32 CTAs an SM of 256 threads with 16 elements each (all of either call's rounds), and no whole number
    of rounds; tokens of half a CTA an SM (one round)."""
    at_once, sms = 256 // (H * d // 16), torch.cuda.get_device_properties(0).multi_processor_count
    assert at_once > 1
    return 33 * sms * at_once + 5 * at_once // 2, sms * at_once // 2


def shuffled(rng, T, bs):
    """Slots of T tokens and the blocks there are: whole blocks from their start, from odd and even offsets, in any order, single
    tokens, padding."""
    NB = 2 * T // bs + 40
    slots, n = [], 0
    for blk in rng.permutation(NB):
        kind, first = rng.random(), int(rng.integers(0, bs))
        offs = np.arange(bs) if kind < 0.5 else np.arange(first, bs) if kind < 0.8 else np.array([first]) if kind < 0.85 else rng.permutation(bs)
        pad = -1 - np.zeros(int(rng.integers(1, 3)) if rng.random() < 0.3 else 0, dtype=np.int64)
        slots += [blk * bs + offs, pad]
        n += len(offs) + len(pad)
        if n >= T:
            break
    slots = np.concatenate(slots)[:T]
    assert len(slots) == T
    return slots, NB


@pytest.mark.parametrize("H,d,bs", [(2, 64, 16), (3, 64, 128), (5, 128, 32), (2, 256, 64)])
def test_rounds_are_one_round(H, d, bs):
    T, short = in_rounds(H, d)
    rng = np.random.default_rng(H * d)
    slots, NB = shuffled(rng, T, bs)
    ids = i32(slots)
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.randn(T, 2, H, d, device="cuda", generator=g).bfloat16()
    start = [torch.from_numpy(x).cuda() for x in cache(rng, NB, H, bs, d)]
    one, many = [x.clone() for x in start], [x.clone() for x in start]
    gdn.gdn_cache4_append(kv[:, 0], kv[:, 1], ids, *one)
    for t in range(0, T, short):
        gdn.gdn_cache4_append(kv[t:t + short, 0], kv[t:t + short, 1], ids[t:t + short], *many)
    for a, b, c in zip(one, many, start):
        assert torch.equal(a, b) and not torch.equal(a, c)
    out = torch.full((T + 1, 2, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache4_read(*one, ids, out[:T, 0], out[:T, 1], err=err)
    assert int(err) == 0 and bool((out[T] == 3.0).all()) and bool((out[:T][ids < 0] == 3.0).all())
    live = torch.nonzero(ids >= 0)[:, 0]
    for part in live.split(20000):
        at = ids[part].long()
        pages, where = torch.unique(at // bs, return_inverse=True)
        for z, x in enumerate(co.unpack(*(y[pages] for y in one))):
            assert same_values(out[part, z], x[where, :, at % bs])


@pytest.mark.parametrize("H,d,bs", [(3, 64, 16), (2, 256, 64)])
@pytest.mark.parametrize("ctas", [0.9, 1.1, 2.9, 3.1, 31.5])
def test_around_the_rounds(H, d, bs, ctas):
    """Calls of just under and over one CTA an SM (a second round), three (four rounds), and under 32 (eight)."""
    T = int(ctas * in_rounds(H, d)[1] * 2) + 1
    rng = np.random.default_rng(T)
    slots, NB = shuffled(rng, T, bs)
    ids = i32(slots)
    kv = torch.randn(T, 2, H, d, device="cuda").bfloat16()
    one = [torch.from_numpy(x).cuda() for x in cache(rng, NB, H, bs, d)]
    many, short = [x.clone() for x in one], in_rounds(H, d)[1]
    gdn.gdn_cache4_append(kv[:, 0], kv[:, 1], ids, *one)
    out, parts = torch.full((2, 2, T, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*one, ids, out[0], out[1])
    for t in range(0, T, short):
        gdn.gdn_cache4_append(kv[t:t + short, 0], kv[t:t + short, 1], ids[t:t + short], *many)
        gdn.gdn_cache4_read(*one, ids[t:t + short], parts[0, t:t + short], parts[1, t:t + short])
    assert all(torch.equal(a, b) for a, b in zip(one, many)) and torch.equal(out, parts)
