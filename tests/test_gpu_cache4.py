"""The writer and the read-back of the 4-bit cache on the GPU: bytes against the plain restatement of
tests/_cache4_oracle.py, exactly."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache4_oracle as co

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def same_values(got, want):
    """bf16 holds every value of the format exactly, but for those of 2^128 and above (the largest bf16 number, 1.99 * 2^127, is
    rounded to 4 * 2^126): they are infinite."""
    got, huge = got.double(), want.abs() >= 2.0 ** 128
    want = torch.where(huge, torch.copysign(torch.full_like(want, torch.inf), want), want)
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def cache(rng, NB, H, bs, d):
    return (rng.integers(0, 256, (NB, H, bs, d // 2), dtype=np.uint8), rng.integers(0, 256, (NB, H, bs // 2, d), dtype=np.uint8),
            rng.integers(0, 255, (NB, H, bs, d // 32), dtype=np.uint8), rng.integers(0, 255, (NB, H, bs, d // 32), dtype=np.uint8))


def values(rng, T, H, d):
    x = rng.standard_normal((T, H, d)) * np.exp(rng.standard_normal((T, H, d // 32, 1)) * 3).repeat(32, axis=-1).reshape(T, H, d)
    return torch.from_numpy(x).bfloat16()


def run_append(k, v, slots, arrays):
    T, H, d = k.shape
    both = torch.zeros(T, 2 * H + 1, d, dtype=torch.bfloat16, device="cuda")   # slices of one projection
    both[:, :H], both[:, H:2 * H] = k.cuda(), v.cuda()
    t = [torch.from_numpy(x.copy()).cuda() for x in arrays]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache4_append(both[:, :H], both[:, H:2 * H], i32(slots), *t, err=err)
    torch.cuda.synchronize()
    return t, int(err)


def check_append(k, v, slots, arrays):
    got, err = run_append(k, v, slots, arrays)
    want = co.append(k.float().numpy(), v.float().numpy(), slots, *arrays)
    nan = [want[2] == 255, want[3] == 255]
    for i, (a, b) in enumerate(zip(got, want)):
        a = a.cpu().numpy()
        if i >= 2:
            assert np.array_equal(a, b), i
    kc, vc = (x.cpu().numpy() for x in got[:2])
    gone = nan[0].repeat(16, axis=3)                      # codes of a group with NaN mean nothing
    assert np.array_equal(np.where(gone, 0, kc), np.where(gone, 0, want[0]))
    for odd in (0, 1):
        gone = nan[1][:, :, odd::2].repeat(32, axis=3)
        half = lambda x: (x >> 4 * odd) & 15  # noqa: E731
        assert np.array_equal(np.where(gone, 0, half(vc)), np.where(gone, 0, half(want[1])))
    return got, err


def slots_of(rng, NB, bs, runs):
    """Slots of runs (block order shuffled, tokens of a run in order)."""
    blocks = rng.permutation(NB)
    out = []
    for i, (first, n) in enumerate(runs):
        out += [int(blocks[i]) * bs + first + j for j in range(n)]
    return out


@pytest.mark.parametrize("H,bs,d", [(1, 16, 64), (3, 32, 128), (2, 128, 256), (8, 16, 64), (17, 64, 256), (5, 64, 128)])
def test_append(H, bs, d):
    rng = np.random.default_rng(H * 100 + bs + d)
    runs = [(0, bs), (1, 1), (3, bs - 3), (0, 1), (2, 1), (bs - 1, 1), (5, 4), (4, 2), (7, 8)]
    slots = slots_of(rng, 12, bs, runs)
    slots = [-1] + slots[:4] + [-7] + slots[4:]           # padding
    k, v = values(rng, len(slots), H, d), values(rng, len(slots), H, d)
    _, err = check_append(k, v, slots, cache(rng, 12, H, bs, d))
    assert err == 0


@pytest.mark.parametrize("T", [1, 2, 3])
def test_single_tokens(T):
    rng = np.random.default_rng(T)
    slots = [5 * 16 + 7, 2 * 16 + 8, 2 * 16 + 3][:T]
    check_append(values(rng, T, 2, 256), values(rng, T, 2, 256), slots, cache(rng, 6, 2, 16, 256))


def test_many_tokens_in_turns():
    """A call that takes its tokens in rounds: 5,000 of them, with a last CTA that is not full."""
    rng = np.random.default_rng(9)
    H, bs, d, NB = 1, 16, 64, 700
    free = rng.permutation(NB)
    slots = [int(b) * bs + j for b in free for j in range(bs)][:10007]
    k, v = values(rng, len(slots), H, d), values(rng, len(slots), H, d)
    got, _ = run_append(k, v, slots, cache(rng, NB, H, bs, d))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(2, len(slots), H, d, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*got, i32(slots), out[0], out[1], err=err)
    kk, vv = co.unpack(*got)
    at = torch.as_tensor(slots, device="cuda")
    for z, x in ((0, kk), (1, vv)):
        assert torch.equal(out[z].double(), x[at // bs, :, at % bs])
    # within a step of the values: at most 1 of a group's 7
    for z, x in ((0, k), (1, v)):
        x = x.double().cuda().unflatten(-1, (-1, 32))
        top = x.abs().amax(dim=-1, keepdim=True)
        assert bool(((out[z].double().unflatten(-1, (-1, 32)) - x).abs() <= top * 2 / 7).all())


def test_extremes():
    """Zeros, the smallest and largest bf16 numbers, powers of two around the limit of a group, infinities, NaN."""
    rng = np.random.default_rng(4)
    x = torch.zeros(12, 1, 64)
    x[1, 0, 0], x[1, 0, 33] = 2.0 ** -133, 2.0 ** -70
    x[2, 0, :2] = torch.tensor([3.3895e38, -3.3895e38])
    x[3, 0, 0], x[3, 0, 32] = 7.0, 7.03125
    x[4, 0, 0], x[4, 0, 32] = 1.75 * 2.0 ** -63, 1.7578125 * 2.0 ** -63
    x[5, 0, 0], x[5, 0, 1], x[5, 0, 40] = torch.inf, 2.0, -torch.inf
    x[6, 0, 5], x[6, 0, 40] = torch.nan, 1.0
    x[7, 0, 5], x[7, 0, 6] = torch.nan, torch.inf
    x[8, 0] = torch.linspace(-7, 7, 64)
    x[9, 0] = -0.0
    x[10, 0, ::2] = 2.5
    x[11, 0] = torch.arange(64) * 0.25
    x = x.bfloat16()
    slots = list(range(16, 28))
    got, _ = check_append(x, x.flip(0), slots, cache(rng, 3, 1, 16, 64))
    out = torch.empty(2, 12, 1, 64, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*got, i32(slots), out[0], out[1])
    k, v = co.unpack(*got)
    for z, want in ((0, k), (1, v)):
        want = want[1, :, :12].transpose(0, 1)
        assert same_values(out[z], want)
    assert bool(torch.isnan(out[0, 6, 0, :32]).all()) and not bool(torch.isnan(out[0, 6, 0, 32:]).any())


def test_every_byte_reads_exactly():
    """All 16 codes under all 256 scales, keys and values, both halves of a byte."""
    NB, bs, d = 16, 16, 64
    ks = torch.arange(256, dtype=torch.uint8).reshape(NB, 1, bs, 1).repeat(1, 1, 1, 2)
    codes = torch.arange(64, dtype=torch.uint8) % 16
    kc = (codes[0::2] | codes[1::2] << 4).repeat(NB, 1, bs, 1)
    vc = (codes | codes.flip(0) << 4).repeat(NB, 1, bs // 2, 1)
    arrays = [x.contiguous().cuda() for x in (kc, vc, ks, ks)]
    slots = i32(np.random.default_rng(0).permutation(256))
    out = torch.empty(2, 256, 1, d, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*arrays, slots, out[0], out[1])
    for z, want in enumerate(co.unpack(*arrays)):
        want = want[slots.long() // bs, :, slots.long() % bs]
        assert same_values(out[z], want)


def test_slots_that_are_not_there_and_rows_that_stay():
    rng = np.random.default_rng(8)
    arrays = cache(rng, 4, 2, 32, 128)
    slots = [3, 4 * 32, -1, 40, 1 << 30, 41]
    k, v = values(rng, 6, 2, 128), values(rng, 6, 2, 128)
    got, err = check_append(k, v, slots, arrays)
    assert err == gdn.GDN_DEVERR_BLOCK_RANGE
    wide = torch.full((6, 5, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache4_read(*got, i32(slots), wide[:, :2], wide[:, 2:4], err=e)
    assert int(e) == gdn.GDN_DEVERR_BLOCK_RANGE
    kk, vv = co.unpack(*got)
    for t, s in enumerate(slots):
        if 0 <= s < 128:
            assert torch.equal(wide[t, :2].double(), kk[s // 32, :, s % 32]) and torch.equal(wide[t, 2:4].double(), vv[s // 32, :, s % 32])
        else:
            assert bool((wide[t] == 7.0).all())
    assert bool((wide[:, 4] == 7.0).all())
    # the same slot twice, in any order
    twice = torch.empty(2, 3, 2, 128, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*got, i32([41, 3, 41]), twice[0], twice[1])
    assert torch.equal(twice[:, 0], twice[:, 2]) and torch.equal(twice[0, 1], wide[0, :2])


def test_written_again_after_speculation():
    """Tokens taken back and written anew: nothing of the first writing stays, and the tokens before are as they were."""
    rng = np.random.default_rng(5)
    arrays = cache(rng, 2, 2, 16, 64)
    a, b = values(rng, 9, 2, 64), values(rng, 9, 2, 64)
    got, _ = run_append(a, a, list(range(16, 25)), arrays)
    once = [x.cpu().numpy() for x in got]
    got, _ = run_append(b[:4], b[:4], [21, 22, 23, 24], once)
    want = co.append(b[:4].float().numpy(), b[:4].float().numpy(), [21, 22, 23, 24], *once)
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(got, want))


def test_a_large_cache():
    """Addresses past 2^32 bytes: the last blocks of a cache of 4.6 GB."""
    NB, H, bs, d = 70000, 4, 128, 256
    kc = torch.zeros(NB, H, bs, d // 2, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(NB, H, bs // 2, d, dtype=torch.uint8, device="cuda")
    ks, vs = torch.zeros(2, NB, H, bs, d // 32, dtype=torch.uint8, device="cuda")
    assert kc.numel() > 1 << 32
    x = values(np.random.default_rng(1), 5, H, d).cuda()
    slots = i32([(NB - 1) * bs + j for j in (3, 4, 5, 127)] + [(NB - 3) * bs])
    gdn.gdn_cache4_append(x, x, slots, kc, vc, ks, vs)
    out = torch.empty(2, 5, H, d, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(kc, vc, ks, vs, slots, out[0], out[1])
    assert torch.equal(out[0], out[1]) and int((kc != 0).any(dim=3).any(dim=1).sum()) == 5
    k, v = co.unpack(kc[-3:], vc[-3:], ks[-3:], vs[-3:])
    assert torch.equal(out[0, 0].double(), k[2, :, 3]) and torch.equal(out[1, 4].double(), v[0, :, 0])


def test_captured_and_on_a_stream():
    rng = np.random.default_rng(2)
    t = [torch.from_numpy(x).cuda() for x in cache(rng, 4, 2, 16, 128)]
    k = values(rng, 6, 2, 128).cuda()
    slots = i32(range(17, 23))
    out = torch.zeros(2, 6, 2, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: (gdn.gdn_cache4_append(k, k, slots, *t), gdn.gdn_cache4_read(*t, slots, out[0], out[1]))  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    k.copy_(values(rng, 6, 2, 128).cuda())
    graph.replay()
    torch.cuda.synchronize()
    first = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, first) and bool((out[0] != 0).any())


@pytest.mark.parametrize("H,d,bs", [(16, 256, 64), (40, 128, 16)])
def test_long_calls_are_short_ones(H, d, bs):
    """Calls long enough that a thread has several tokens: runs that start at odd and even slots, single tokens, padding and
    any order give the bytes that calls of 50 tokens at a time give, and read back the same."""
    rng = np.random.default_rng(d)
    NB, T = 6000 // bs + 40, 6000
    slots, blocks = [], list(rng.permutation(NB))
    while len(slots) < T:
        blk, kind = int(blocks.pop()), rng.random()
        first = int(rng.integers(0, bs))
        run = list(range(blk * bs + first, blk * bs + bs)) if kind < 0.8 else [blk * bs + int(x) for x in rng.permutation(bs)]
        slots += run + ([-1] if rng.random() < 0.3 else [])
        if len(blocks) == 1:
            break
    slots = slots[:T]
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn(len(slots), 2, H, d, device="cuda", generator=g).bfloat16()
    ids = i32(slots)
    start = [torch.from_numpy(x).cuda() for x in cache(rng, NB, H, bs, d)]
    one, many = [x.clone() for x in start], [x.clone() for x in start]
    gdn.gdn_cache4_append(kv[:, 0], kv[:, 1], ids, *one)
    for t in range(0, len(slots), 50):
        gdn.gdn_cache4_append(kv[t:t + 50, 0], kv[t:t + 50, 1], ids[t:t + 50], *many)
    for a, b in zip(one, many):
        assert torch.equal(a, b)
    assert not torch.equal(one[0], start[0])
    out, parts = torch.full((2, 2, len(slots), H, d), 3.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_cache4_read(*one, ids, out[0], out[1])
    for t in range(0, len(slots), 50):
        gdn.gdn_cache4_read(*one, ids[t:t + 50], parts[0, t:t + 50], parts[1, t:t + 50])
    assert torch.equal(out, parts)
    k, v = co.unpack(*(x[:64] for x in one))
    at = torch.nonzero((ids >= 0) & (ids < 64 * bs))[:, 0]
    assert same_values(out[0, at], k[ids[at].long() // bs, :, ids[at].long() % bs])
    assert same_values(out[1, at], v[ids[at].long() // bs, :, ids[at].long() % bs])


def test_refused_before_the_call():
    rng = np.random.default_rng(1)
    t = [torch.from_numpy(x).cuda() for x in cache(rng, 4, 2, 16, 64)]
    k = values(rng, 3, 2, 64).cuda()
    slots, err = i32([1, 2, 3]), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache4_append(k, k, slots, *t, err=err)
    before = [x.clone() for x in t]
    bad_calls = [lambda: gdn.gdn_cache4_append(k, k, slots.long(), *t), lambda: gdn.gdn_cache4_append(k.float(), k, slots, *t),
                 lambda: gdn.gdn_cache4_append(k, k[:, :1], slots, *t), lambda: gdn.gdn_cache4_append(k, k, slots, *t, err=err.float()),
                 lambda: gdn.gdn_cache4_append(k, k, slots.cpu(), *t), lambda: gdn.gdn_cache4_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, slots, *t),
                 lambda: gdn.gdn_cache4_append(k, k, slots, t[0][:, :, ::2], *t[1:]), lambda: gdn.gdn_cache4_append(k, k, slots, t[0][:2], *t[1:]),
                 lambda: gdn.gdn_cache4_append(k, k, slots, t[0], t[1], t[2], t[3].float()), lambda: gdn.gdn_cache4_append(k, k, None, *t),
                 lambda: gdn.gdn_cache4_read(*t, slots, k, k[:2]), lambda: gdn.gdn_cache4_read(*t, slots, k.view(torch.float16), k)]
    for call in bad_calls:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gdn.GDNError):                       # a row that does not start on 16 bytes
        flat = torch.zeros(3 * 128 + 8, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_cache4_append(flat[4:4 + 384].view(3, 2, 64), k, slots, *t)
    assert all(torch.equal(x, y) for x, y in zip(t, before))
