"""The paged 8-bit cache on the GPU: its tables, its writer and the attention over it, against the
plain restatements of tests/_cache_oracle.py. Tables and bytes are compared exactly; attention
within an elementwise bound that follows from what the kernels round (f16 probabilities in the
single-token kernel: 11 bits, 2^-25 below the largest; two e4m3 parts in the prompt kernel: 9 bits,
2^-14 below it)."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache_oracle as co

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------- tables

def run_tables(old, new, table, ring, pool, bs, capacity, in_place=False):
    B = len(old)
    d = {"old": i32(old), "new": i32(new), "table": i32(table), "ring": i32(ring), "pool": i32(pool)}
    out = d["pool"] if in_place else torch.full((2,), -7, dtype=torch.int32, device="cuda")
    lens = d["old"] if in_place else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    cu = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((capacity,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((capacity,), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache_tables(d["old"], d["new"], d["table"], d["ring"], d["pool"], out, cu, slots, pos,
                         lens, bs, err=err)
    torch.cuda.synchronize()
    got = {"table": d["table"], "ring": d["ring"], "pool": out, "cu": cu, "slots": slots,
           "positions": pos, "lens": lens}
    return {k: v.cpu().numpy() for k, v in got.items()}, int(err)


def table_case(seed, B, bs, max_len, max_new, shortage=0):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, max_len + 1, B)
    new = old + rng.integers(0, max_new + 1, B)
    kind = rng.random(B)
    new = np.where(kind < 0.15, 0, np.where(kind < 0.25, old // 2, new))
    old = np.where(kind > 0.85, 0, old)
    n = lambda l: -(-l // bs)  # noqa: E731
    width = int(n(np.maximum(old, new)).max()) + 1
    used = int(n(old).sum())
    need = int(np.maximum(0, n(new) - n(old)).sum())
    total = used + max(need - shortage, 0) + (0 if shortage else 5) + 1
    perm = rng.permutation(total)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :n(old[b])] = perm[at:at + n(old[b])]
        at += n(old[b])
    free = perm[used:]
    head = int(rng.integers(0, total))
    ring = np.full(total, -1)
    ring[(head + np.arange(free.size)) % total] = free
    return old, new, table, ring, np.array([head, free.size])


@pytest.mark.parametrize("B,bs,max_len,max_new,spare", [
    (1, 16, 0, 1, 0), (1, 128, 1000, 300, 3), (7, 32, 200, 1, 0), (64, 64, 8192, 1, 2),
    (513, 16, 300, 40, 11), (1500, 16, 90, 5, 0), (40, 128, 700, 900, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(B, bs, max_len, max_new, spare, in_place):
    old, new, table, ring, pool = table_case(B * 31 + bs, B, bs, max_len, max_new)
    T = int(np.maximum(0, new - old).sum()) + spare
    want = co.tables(old, new, table, ring, pool, bs, T)
    got, err = run_tables(old, new, table, ring, pool, bs, T, in_place)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert err == 0 and not want["bad"] and not want["short"]


@pytest.mark.parametrize("B,shortage", [(3, 1), (100, 7), (700, 400)])
def test_tables_short_of_blocks(B, shortage):
    """Rows are served in order until the free blocks run out; the rest keep their length."""
    old, new, table, ring, pool = table_case(B, B, 16, 200, 60, shortage)
    T = int(np.maximum(0, new - old).sum())
    want = co.tables(old, new, table, ring, pool, 16, T)
    assert want["short"] or B == 3     # (the smallest case happens to need no block)
    got, err = run_tables(old, new, table, ring, pool, 16, T)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert err == (gdn.GDN_DEVERR_BLOCKS if want["short"] else 0)


def test_tables_bad_lengths_capacity_and_pool():
    old, new, table, ring, pool = table_case(5, 20, 32, 100, 30)
    old[3], new[7] = -1, table.shape[1] * 32 + 1
    T = int(sum(max(0, w - o) for i, (o, w) in enumerate(zip(old, new)) if i not in (3, 7)))
    want = co.tables(old, new, table, ring, pool, 32, T)
    got, err = run_tables(old, new, table, ring, pool, 32, T)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert err == gdn.GDN_DEVERR_SEQLENS
    old, new, table, ring, pool = table_case(6, 20, 32, 100, 30)
    want = co.tables(old, new, table, ring, pool, 32, 10)      # more tokens than slots
    got, err = run_tables(old, new, table, ring, pool, 32, 10)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert err == gdn.GDN_DEVERR_SEQLENS
    got, err = run_tables(old, new, table, ring, [ring.size, 3], 32, 10)   # no such head
    assert err & gdn.GDN_DEVERR_BLOCKS and got["pool"][1] >= 0


# ------------------------------------------------------------------------------------- writer

def run_append(k, v, slots, kc, vc, ks, vs):
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    T, H, d = k.shape
    both = torch.zeros(T, 2 * H + 1, d, dtype=torch.bfloat16, device="cuda")   # slices of one projection
    both[:, :H], both[:, H:2 * H] = dev(k).bfloat16(), dev(v).bfloat16()
    t = [dev(kc), dev(vc), dev(ks), dev(vs)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache_append(both[:, :H], both[:, H:2 * H], i32(slots), *t, err=err)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in t], int(err)


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def same_bytes(a, b):
    """Equal bytes, any NaN standing for any other."""
    nan = lambda x: (x & 127) == 127  # noqa: E731
    return np.array_equal(np.where(nan(a), 127, a), np.where(nan(b), 127, b))


@pytest.mark.parametrize("d,bs,H", [(64, 16, 1), (64, 128, 3), (128, 32, 2), (256, 64, 2), (256, 128, 1), (128, 16, 5)])
@pytest.mark.parametrize("runs", ["one token each", "prompts", "mixed"])
def test_append(d, bs, H, runs):
    rng = np.random.default_rng(d + bs + H)
    NB = 40
    cache = lambda: rng.integers(0, 256, (NB, H, bs, d)).astype(np.uint8)  # noqa: E731
    scale = lambda: np.exp2(rng.uniform(-12, 2, (NB, H))).astype(np.float32)  # noqa: E731
    kc, vc, ks, vs = cache(), cache(), scale(), scale()
    blocks = list(rng.permutation(NB))
    slots = []
    for i in range(30 if runs != "prompts" else 9):
        long = runs == "prompts" or (runs == "mixed" and i % 3 == 0)
        left = int(rng.integers(1, 3 * bs)) if long else 1
        off = int(rng.integers(0, bs)) if i % 4 else 0
        while left and blocks:
            n = min(left, bs - off)
            b = int(blocks.pop())
            slots += [b * bs + off + j for j in range(n)]
            left, off = left - n, 0
        if i % 5 == 2:
            slots += [-1]
    slots = np.array(slots)
    size = np.exp2(rng.uniform(-10, 6, (len(slots), 1, 1)))
    k, v = (bf16(rng.standard_normal((len(slots), H, d)) * size) for _ in range(2))
    (gk, gv, gks, gvs), err = run_append(k, v, slots, kc, vc, ks, vs)
    for x, c, s, gc, gs in ((k, kc, ks, gk, gks), (v, vc, vs, gv, gvs)):
        wc, ws = co.append(x, slots, c, s)
        assert np.array_equal(gs, ws)
        assert same_bytes(gc, wc)
    assert err == 0


def test_append_special_values():
    """Zeros, infinities, NaN, the smallest and largest bf16, exact ties of the rounding."""
    H, d, bs, NB = 2, 64, 16, 6
    x = np.zeros((20, H, d), np.float32)
    x[1, 0, :5] = [np.inf, -np.inf, np.nan, 1.0, -3.0]
    x[2:5, 0] = 2.0 ** -133
    x[5, 1] = 3.3895e38
    x[6, 1, 0] = np.nan
    x[16, 0] = 448.0 * np.linspace(-1, 1, d)
    x[17, 0, :8] = [17, 18.0, 19, 21, 23, 0.00146484375, 0.0009765625, 0.0029296875]
    x[18, 0] = np.nan
    x[19, 1] = np.inf
    x = bf16(x)
    slots = np.concatenate([np.arange(16) + 2 * bs, np.array([5 * bs, 5 * bs + 1, 0, bs + 3])])
    kc = np.random.default_rng(0).integers(0, 256, (NB, H, bs, d)).astype(np.uint8)
    ks = np.full((NB, H), 0.01, np.float32)
    (gk, _, gks, _), err = run_append(x, x, slots, kc, kc, ks, ks)
    wc, ws = co.append(x, slots, kc, ks)
    assert np.array_equal(gks, ws) and same_bytes(gk, wc) and err == 0


def test_append_token_by_token_grows_the_scale():
    """A block filled in 16 calls: each step's bytes and scales as the definition's."""
    H, d, bs = 2, 128, 16
    rng = np.random.default_rng(3)
    kc, ks = np.zeros((3, H, bs, d), np.uint8), np.zeros((3, H), np.float32)
    vc, vs = kc.copy(), ks.copy()
    for i in range(bs):
        x = bf16(rng.standard_normal((1, H, d)) * 1.5 ** i)
        y = bf16(rng.standard_normal((1, H, d)) * 0.7 ** i)
        want = co.append(x, [bs + i], kc, ks), co.append(y, [bs + i], vc, vs)
        (kc, vc, ks, vs), _ = run_append(x, y, [bs + i], kc, vc, ks, vs)
        assert same_bytes(kc, want[0][0]) and np.array_equal(ks, want[0][1])
        assert same_bytes(vc, want[1][0]) and np.array_equal(vs, want[1][1])


def test_append_slots_outside_the_cache():
    H, d, bs, NB = 1, 64, 32, 2
    x = bf16(np.random.default_rng(1).standard_normal((4, H, d)))
    kc, ks = np.zeros((NB, H, bs, d), np.uint8), np.ones((NB, H), np.float32)
    slots = [NB * bs, -5, 3, 2 ** 31 - 1]
    (gk, gv, gks, gvs), err = run_append(x, x, slots, kc, kc, ks, ks)
    wc, ws = co.append(x, slots, kc, ks)
    assert np.array_equal(gk, wc) and np.array_equal(gks, ws) and np.array_equal(gv, wc)
    assert err == gdn.GDN_DEVERR_BLOCK_RANGE


# ---------------------------------------------------------------------------------- attention

class Cache:
    """A random cache with shuffled pages. Bytes past a request's length, and the pages that no
    request holds, are NaN."""

    def __init__(self, seed, lens, H, d, bs, spread=1.0, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        n = [-(-max(int(l), 0) // bs) for l in lens]
        NB = sum(n) + 3
        W = width or max(n + [1]) + 1
        perm = rng.permutation(NB)
        table = np.full((len(lens), W), -1)
        at = 0
        for b, x in enumerate(n):
            table[b, :x] = perm[at:at + x]
            at += x

        def pool():
            x = (torch.randn(NB, H, bs, d, device="cuda", generator=g) * 60).clamp(-448, 448)
            x = x.to(co.F8).view(torch.uint8)
            s = torch.exp2(spread * torch.randn(NB, H, device="cuda", generator=g)) / 60
            return x, s

        self.kc, self.ks = pool()
        self.vc, self.vs = pool()
        for b, l in enumerate(lens):
            if l > 0 and l % bs:
                last = int(table[b, n[b] - 1])
                self.kc[last, :, l % bs:] = 0x7F
                self.vc[last, :, l % bs:] = 0xFF
        for f in perm[sum(n):]:
            self.kc[int(f)] = 0x7F
            self.vc[int(f)] = 0x7F
        self.table, self.lens = i32(table), i32(lens)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = (H, d, bs)

    def pools(self):
        return self.kc, self.vc, self.ks, self.vs


def queries(seed, T, Hq, d, size=1.0, strided=False):
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    q = (torch.randn(T, Hq + (2 if strided else 0), d, device="cuda", generator=g) * size).bfloat16()
    return q[:, :Hq]


def decode(c, q, scale=None, rows=None, stream=None):
    table, lens = (c.table, c.lens) if rows is None else (c.table[rows].contiguous(), c.lens[rows].contiguous())
    H, d, bs = c.dims
    ws = torch.full((gdn.gdn_attn_decode_workspace_size(q.shape[0], table.shape[1], q.shape[1], H, d, bs),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((q.shape[0], q.shape[1], d), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_attn_decode(q, *c.pools(), table, lens, out, ws, scale=scale, err=c.err, stream=stream)
    return out


def prefill(c, q, cu, scale=None, rows=None):
    table, lens = (c.table, c.lens) if rows is None else (c.table[rows].contiguous(), c.lens[rows].contiguous())
    H, d, bs = c.dims
    ws = torch.full((gdn.gdn_attn_prefill_workspace_size(q.shape[0], lens.shape[0], table.shape[1], q.shape[1], H, d, bs),),
                    0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((q.shape[0], q.shape[1], d), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_attn_prefill(q, i32(cu), *c.pools(), table, lens, out, ws, scale=scale, err=c.err)
    return out


def check(out, want, tol):
    assert bool(torch.isfinite(out.float()).all())
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


DECODE = dict(p_bits=11, p_floor=2.0 ** -25)
PREFILL = dict(p_bits=9, p_floor=2.0 ** -13)   # 2^-14 relative to a vs_ref that may be 1.75 times too large


@pytest.mark.parametrize("Hq,H,d,bs", [
    (16, 2, 256, 64), (32, 8, 128, 16), (28, 4, 64, 32), (3, 3, 128, 128), (9, 1, 256, 16), (16, 1, 128, 64),
    (20, 1, 64, 16), (34, 2, 256, 32), (5, 5, 64, 128), (12, 1, 64, 64)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 15, 16, 17, 129, 0], [255, 256, 257, 700, 1024, 1025], [4097, 33, 8193]])
def test_attn_decode(Hq, H, d, bs, lens):
    c = Cache(Hq + d + bs + len(lens), lens, H, d, bs)
    q = queries(len(lens), len(lens), Hq, d, strided=True)
    out = decode(c, q)
    want, tol = co.attention(q, None, *c.pools(), c.table, lens, d ** -0.5, **DECODE)
    check(out, want, tol)
    assert int(c.err) == 0


@pytest.mark.parametrize("Hq,H,d,bs", [
    (16, 2, 256, 64), (32, 8, 128, 16), (28, 4, 64, 32), (3, 3, 128, 128), (9, 1, 256, 16), (34, 2, 64, 16)])
@pytest.mark.parametrize("new,old", [
    ([1], [0]), ([5, 1, 130, 0, 17], [0, 40, 3, 9, 500]), ([257, 64], [0, 1000]), ([3], [5000]), ([33, 2], [2100, 4096])])
def test_attn_prefill(Hq, H, d, bs, new, old):
    lens = [a + b for a, b in zip(new, old)]
    c = Cache(Hq + d + bs + len(new), lens, H, d, bs)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = queries(d, int(cu[-1]) + 3, Hq, d, strided=True)
    out = prefill(c, q, cu)
    want, tol = co.attention(q, cu, *c.pools(), c.table, lens, d ** -0.5, **PREFILL)
    check(out[:cu[-1]], want[:cu[-1]], tol[:cu[-1]])
    assert bool((out[cu[-1]:] == 7.0).all())     # rows past the step's tokens are not written
    assert int(c.err) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size,scale,spread", [(1.0, None, 6.0), (30.0, None, 1.0), (1.0, -0.2, 1.0), (1e-3, 0.0, 1.0),
                                               (2e4, 2e-5, 2.0)])
def test_attn_scales_and_sizes(d, size, scale, spread):
    """Blocks whose scales differ by many powers of two, sharp and flat softmax, odd `scale`s."""
    lens, Hq, H = [700, 90, 1300], 8, 2
    c = Cache(d + 1, lens, H, d, 16, spread=spread)
    sc = d ** -0.5 if scale is None else scale
    q = queries(4, 3, Hq, d, size)
    want, tol = co.attention(q, None, *c.pools(), c.table, lens, sc, **DECODE)
    check(decode(c, q, scale), want, tol)
    cu = [0, 40, 41, 100]
    q = queries(5, 100, Hq, d, size)
    want, tol = co.attention(q, cu, *c.pools(), c.table, lens, sc, **PREFILL)
    check(prefill(c, q, cu, scale), want, tol)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_rows_that_see_nothing(d):
    """Lengths shorter than the new tokens (a refused row): the first tokens see no key."""
    new, lens = [6, 40, 3], [4, 0, 3]
    c = Cache(d, lens, 2, d, 16)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = queries(1, int(cu[-1]), 6, d)
    out = prefill(c, q, cu)
    want, tol = co.attention(q, cu, *c.pools(), c.table, lens, d ** -0.5, **PREFILL)
    check(out, want, tol)
    assert bool((out[:2] == 0).all()) and bool((out[6:46] == 0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_blocks_that_are_none(d):
    """A table entry outside the cache: its tokens are not seen, the error word says so."""
    lens = [300, 200]
    c = Cache(d + 2, lens, 2, d, 32)
    c.table[0, 3], c.table[1, 0] = -4, c.kc.shape[0]
    q = queries(2, 2, 8, d)
    want, tol = co.attention(q, None, *c.pools(), c.table, lens, d ** -0.5, **DECODE)
    check(decode(c, q), want, tol)
    assert int(c.err) == gdn.GDN_DEVERR_BLOCK_RANGE
    c.err.zero_()
    cu = [0, 150, 200]
    q = queries(3, 200, 8, d)
    want, tol = co.attention(q, cu, *c.pools(), c.table, lens, d ** -0.5, **PREFILL)
    check(prefill(c, q, cu), want, tol)
    assert int(c.err) == gdn.GDN_DEVERR_BLOCK_RANGE
    c.table[:] = -1
    assert bool((prefill(c, q, cu) == 0).all()) and bool((decode(c, q[:2]) == 0).all())


def test_attn_lengths_and_ranges_out_of_bounds():
    c = Cache(1, [40, 50, 60], 2, 128, 16, width=4)     # capacity 64
    c.lens.copy_(i32([-3, 1000, 60]))
    q = queries(1, 3, 4, 128)
    c.table[1] = c.table[2]
    out = decode(c, q)
    assert int(c.err) == gdn.GDN_DEVERR_SEQLENS
    assert bool((out[0] == 0).all())
    c.err.zero_()
    out = prefill(c, q, [0, 1, 2, 4])                   # the third range ends past the rows
    assert int(c.err) == gdn.GDN_DEVERR_SEQLENS
    assert bool((out[2] == 7.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_non_finite_queries_stay_in_their_row(d):
    lens = [100, 900]
    c = Cache(d, lens, 1, d, 16)
    q = queries(1, 2, 4, d)
    clean = decode(c, q)
    q[0, 1, 3], q[1, 2, 0] = float("nan"), float("inf")
    out = decode(c, q)
    assert bool(out[0, 1].isnan().all()) and bool(out[1, 2].isnan().all())
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = keep[1, 2] = False
    assert torch.equal(out[keep], clean[keep])
    cu = [0, 50, 53]
    q = queries(2, 53, 4, d)
    clean = prefill(c, q, cu)
    q[7, 1, 3], q[51, 2, 0] = float("nan"), float("-inf")
    out = prefill(c, q, cu)
    keep = torch.ones(53, 4, dtype=torch.bool)
    keep[7, 1] = keep[51, 2] = False
    assert bool(out[7, 1].isnan().all()) and bool(out[51, 2].isnan().all())
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("Hq,H,d", [(16, 2, 256), (8, 4, 128), (6, 1, 64)])
def test_attn_does_not_depend_on_the_batch(Hq, H, d):
    """A request's result, bit for bit, alone and among others, and from run to run."""
    lens = [5, 4300, 700, 0, 9000, 260, 1]
    c = Cache(d, lens, H, d, 32)
    q = queries(3, len(lens), Hq, d)
    out = decode(c, q)
    assert torch.equal(out, decode(c, q))
    for b in (1, 2, 4, 6):
        assert torch.equal(out[b:b + 1], decode(c, q[b:b + 1], rows=[b]))
    new = [3, 20, 300, 0, 2, 260, 1]
    cu = np.concatenate([[0], np.cumsum(new)])
    q = queries(4, int(cu[-1]), Hq, d)
    out = prefill(c, q, cu)
    assert torch.equal(out, prefill(c, q, cu))
    for b in (1, 2, 4, 6):
        one = prefill(c, q[cu[b]:cu[b + 1]], [0, new[b]], rows=[b])
        assert torch.equal(out[cu[b]:cu[b + 1]], one)


def test_attn_many_requests():
    """More requests than one launch holds, most of them short."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 4500)
    c = Cache(8, lens, 1, 64, 16)
    q = queries(6, 4500, 2, 64)
    want, tol = co.attention(q, None, *c.pools(), c.table, lens, 0.125, **DECODE)
    check(decode(c, q), want, tol)
    want, tol = co.attention(q, np.arange(4501), *c.pools(), c.table, lens, 0.125, **PREFILL)
    check(prefill(c, q, np.arange(4501)), want, tol)


def test_step_on_another_stream_and_in_a_graph():
    """Tables, writer and attention of two steps on a side stream, captured and replayed; the
    cache then holds what the tokens were, to 8 bits."""
    B, H, Hq, d, bs, NB = 5, 2, 6, 128, 16, 64
    lens0 = [0, 3, 31, 16, 47]
    new = [20, 1, 1, 1, 5]
    n = [-(-l // bs) for l in lens0]
    table = np.full((B, 8), -1)
    at = 0
    for b in range(B):
        table[b, :n[b]] = np.arange(at, at + n[b])
        at += n[b]
    ring = np.concatenate([np.arange(at, NB), np.full(at, -1)])
    T = sum(new)
    s = {"old": i32(lens0), "new": i32(np.add(lens0, new)), "table": i32(table), "ring": i32(ring), "pool": i32([0, NB - at]),
         "pool2": i32([0, 0]), "cu": i32(np.zeros(B + 1)), "slots": i32(np.zeros(T)), "pos": i32(np.zeros(T)), "lens": i32(np.zeros(B))}
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.randint(0, 120, (NB, H, bs, d), device="cuda", generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 120, (NB, H, bs, d), device="cuda", generator=g, dtype=torch.uint8)
    ks = torch.full((NB, H), 0.01, device="cuda")
    vs = torch.full((NB, H), 0.01, device="cuda")
    k, v = (torch.randn(T, H, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = queries(9, T, Hq, d)
    out = torch.zeros_like(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdn_attn_prefill_workspace_size(T, B, 8, Hq, H, d, bs), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        gdn.gdn_cache_tables(s["old"], s["new"], s["table"], s["ring"], s["pool"], s["pool2"], s["cu"], s["slots"], s["pos"],
                             s["lens"], bs, err=err)
        gdn.gdn_cache_append(k, v, s["slots"], kc, vc, ks, vs, err=err)
        gdn.gdn_attn_prefill(q, s["cu"], kc, vc, ks, vs, s["table"], s["lens"], out, ws, err=err)

    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and int(err) == 0
    lens = s["lens"].tolist()
    assert lens == list(np.add(lens0, new))
    want, tol = co.attention(q, s["cu"].tolist(), kc, vc, ks, vs, s["table"], lens, d ** -0.5, **PREFILL)
    check(out, want, tol)
    back = kc.view(co.F8).float()[(s["slots"] // bs).long(), :, (s["slots"] % bs).long()] * ks[(s["slots"] // bs).long()][:, :, None]
    assert bool(((back - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + ks.max() * 2.0 ** -9).all())
