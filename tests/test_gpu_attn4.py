"""Attention over the 4-bit cache on the GPU, single tokens and prompts, against the 64-bit restatement of
tests/_cache4_oracle.py, within an elementwise bound that follows from what the kernels round."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache4_oracle as co

pytestmark = pytest.mark.gpu

# What is rounded (include/gdn.h): single tokens: probabilities to f16 (half a step 2^-11), from 2^-34 of the largest. Prompts:
# 11 significant bits (half a step 2^-11), and 2^-32 (2^-28 at 256) of the largest; values of a block below 2^-14 of its
# largest scale to 2^-18 of its largest value.
ROUNDING = {"decode": lambda d: dict(p_bits=11, p_floor=2.0 ** -34),
            "prefill": lambda d: dict(p_bits=11, p_floor=2.0 ** (-28 if d == 256 else -32), k_off=2.0 ** -18, v_off=2.0 ** -18)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


class Case:
    """A cache with shuffled pages, requests of the given lengths and new tokens."""

    def __init__(self, seed, new, old, Hq, H, d, bs, *, spread=3, q_size=1.5, slack=0):
        g = torch.Generator().manual_seed(seed)
        self.new, lens = list(new), [n + o for n, o in zip(new, old)]
        n = [-(-x // bs) for x in lens]
        NB = sum(n) + 4
        self.heads, self.bs, self.W = (Hq, H, d), bs, max(n + [1]) + 1
        perm = torch.randperm(NB, generator=g)
        table = torch.full((len(lens), self.W), -1)
        at = 0
        for b, x in enumerate(n):
            table[b, :x] = perm[at:at + x]
            at += x
        byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
        scale = lambda: torch.randint(127 - spread, 128, (NB, H, bs, d // 32), generator=g, dtype=torch.uint8).cuda()  # noqa: E731
        self.cache = [byte(NB, H, bs, d // 2), byte(NB, H, bs // 2, d), scale(), scale()]
        self.T = sum(new)
        self.q = (q_size / d ** 0.5 * torch.randn(self.T + slack, Hq, d, generator=g)).bfloat16().cuda()
        self.table, self.lens = table.int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.blocks = sum(n)

    def decode(self, q=None, out=None, ws=None, **kw):
        q = self.q if q is None else q
        Hq, H, d = self.heads
        out = torch.full_like(q, 5.0, memory_format=torch.contiguous_format) if out is None else out
        if ws is None:
            ws = torch.empty(gdn.gdn_attn4_decode_workspace_size(q.shape[0], self.W, Hq, H, d, self.bs), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn4_decode(q, *self.cache, self.table, self.lens, out, ws, err=self.err, **kw)
        return out

    def prefill(self, q=None, out=None, ws=None, held=None, **kw):
        q = self.q if q is None else q
        Hq, H, d = self.heads
        out = torch.full_like(q, 5.0, memory_format=torch.contiguous_format) if out is None else out
        if ws is None:
            ws = torch.empty(gdn.gdn_attn4_prefill_workspace_size(q.shape[0], len(self.new), self.W, Hq, H, d, self.bs, held_blocks=held),
                             dtype=torch.uint8, device="cuda")
        gdn.gdn_attn4_prefill(q, self.cu, *self.cache, self.table, self.lens, out, ws, held_blocks=held, err=self.err, **kw)
        return out

    def check(self, got, which, scale=None, q=None, v_exp=0):
        d = self.heads[2]
        k, v = co.unpack(*self.cache)
        cu = None if which == "decode" else self.cu.tolist()
        want, tol = co.attention(self.q if q is None else q, cu, k, v, self.table, self.lens, d ** -0.5 if scale is None else scale,
                                 v_exp=v_exp, **ROUNDING[which](d))
        off = (got.double() - want).abs()
        assert bool((off <= tol).all()), float((off / tol).max())


# ------------------------------------------------------------------------------------- single tokens

@pytest.mark.parametrize("Hq,H,d,bs", [(1, 1, 64, 16), (4, 1, 64, 128), (14, 2, 64, 16), (16, 1, 64, 32), (3, 3, 128, 32), (28, 4, 128, 16),
                                       (8, 1, 128, 64), (32, 2, 128, 128), (18, 1, 128, 16), (16, 2, 256, 64), (8, 8, 256, 16), (32, 2, 256, 32),
                                       (12, 1, 256, 128), (35, 1, 256, 64)])
def test_decode(Hq, H, d, bs):
    """Lengths of a unit, around it and far beyond, ragged; groups of one head to several chunks of 16."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 255, 256, 257, 300, 1000, 2049, 0]
    c = Case(Hq * 1000 + d + bs, [1] * len(lens), [x - 1 if x else -1 for x in lens], Hq, H, d, bs)
    got = c.decode()
    c.check(got, "decode")
    assert int(c.err) == 0 and bool((got[-1] == 0).all())


@pytest.mark.parametrize("Hq,H,d,bs,lens", [(16, 2, 256, 64, [6144, 6145, 12288, 12289, 1]), (4, 1, 64, 16, [24 * 512 + 1, 40000, 33]),
                                            (16, 1, 128, 128, [70001])])
def test_decode_long(Hq, H, d, bs, lens):
    """Units of every size, joined in order by one thread and by rows of them."""
    c = Case(d, [1] * len(lens), [x - 1 for x in lens], Hq, H, d, bs)
    c.check(c.decode(), "decode")


def test_decode_many_units():
    """More units than the join keeps weights of at a time: 1,100 of 1,024 keys, in pages that requests share."""
    c = Case(3, [1], [4095], 2, 1, 64, 128)
    one = c.table[:, :32]
    c.table = one.repeat(1, 1100 * 8 // 32 + 1).contiguous()
    c.W, n = c.table.shape[1], 1100 * 1024 - 5
    c.lens[:] = n
    got = c.decode()
    # the same 4,096 keys 275 times over, but for the last five
    k, v = co.unpack(*c.cache)
    keys, vals = (x[one[0].long(), 0].reshape(-1, 64) for x in (k, v))
    s = c.q[0].double() @ keys.T / 8
    p = torch.exp(s - s.amax(dim=1, keepdim=True)) * torch.where(torch.arange(4096, device="cuda") < 4091, 275.0, 274.0)
    want = p @ vals / p.sum(dim=1, keepdim=True)
    mag = p @ vals.abs() / p.sum(dim=1, keepdim=True)
    assert bool(((got[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + n * 2.0 ** -23) * mag).all())


def test_decode_batches_of_more_than_a_launch():
    lens = [(i * 37) % 400 for i in range(700)]
    c = Case(11, [1] * 700, [x - 1 if x else -1 for x in lens], 4, 2, 64, 16)
    got = c.decode()
    c.check(got, "decode")


def test_decode_strides_scale_and_sign():
    c = Case(5, [1] * 6, [5, 99, 300, 16, 0, 700], 8, 2, 128, 32)
    wide = torch.randn(6, 13, 128, device="cuda").bfloat16()
    for scale in (0.3, -0.2, 0.0):
        got = c.decode(q=wide[:, 2:10], scale=scale)
        c.check(got, "decode", scale=scale, q=wide[:, 2:10])


@pytest.mark.parametrize("Hq,H,d", [(4, 2, 64), (12, 1, 128), (16, 2, 256)])
def test_rows_do_not_depend_on_the_batch(Hq, H, d):
    lens = [1, 40, 257, 1500, 6200, 700, 128]
    c = Case(21, [1] * len(lens), [x - 1 for x in lens], Hq, H, d, 64)
    all_, table, ls, q = c.decode(), c.table, c.lens, c.q
    for pick in ([3], [6, 4], [2, 5, 1, 0], [4, 4, 4]):
        c.table, c.lens = table[pick].contiguous(), ls[pick].contiguous()
        assert torch.equal(c.decode(q=q[pick].contiguous()), all_[pick])
    c.table, c.lens = torch.nn.functional.pad(table, (0, 900), value=-1).contiguous(), ls     # a longer table: another grid
    c.W = c.table.shape[1]
    assert torch.equal(c.decode(), all_)


# --------------------------------------------------------------------- what no request sees, and bad tables

@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("d,H,G", [(64, 2, 4), (128, 1, 9), (256, 2, 8)])
def test_bytes_past_the_length_do_nothing(which, d, H, G):
    """NaN scales, the largest scales and any codes behind a request's last token, in its pages and in others."""
    new = [1, 1, 1, 1] if which == "decode" else [7, 1, 30, 20]
    c = Case(31, new, [20, 64, 300, 0], H * G, H, d, 32)
    run = getattr(c, which)
    clean = run()
    c.check(clean, which)
    used = torch.zeros(c.cache[2].shape[0], c.bs, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens.tolist()):
        for p in range(n):
            used[c.table[b, p // c.bs].long(), p % c.bs] = True
    for fill in (255, 254, 0):
        for x in c.cache[2:]:
            x.copy_(torch.where(used[:, None, :, None], x, fill))
        assert torch.equal(run(), clean), fill
    c.cache[0].copy_(torch.where(used[:, None, :, None], c.cache[0], 0x77))
    half = used.reshape(-1, c.bs // 2, 2)[:, None, :, None, :]
    was = c.cache[1]
    c.cache[1] = torch.where(half[..., 0], was & 15, 7) | torch.where(half[..., 1], was & 240, 0xF0)
    assert torch.equal(run(), clean)


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (128, 16, 1), (256, 16, 2)])
def test_pages_that_are_none(which, d, Hq, H):
    """Holes in a table are not seen; a request of none but holes gives zeros."""
    new = [1, 1, 1] if which == "decode" else [5, 40, 3]
    c = Case(41, new, [200, 300, 90], Hq, H, d, 16)
    c.table[0, 3] = -1
    c.table[0, 7] = c.cache[0].shape[0]
    c.table[1, 0] = 0x7fffffff
    c.table[2] = -5
    got = getattr(c, which)()
    c.check(got, which)
    assert int(c.err) == gdn.GDN_DEVERR_BLOCK_RANGE
    assert bool((got[-1] == 0).all())


def test_lengths_that_are_none():
    c = Case(51, [1, 1, 1], [40, 40, 40], 4, 2, 64, 16)
    good = c.decode()
    assert int(c.err) == 0
    c.lens[1], c.lens[2] = -3, c.W * 16 + 1
    got = c.decode()
    assert int(c.err) & gdn.GDN_DEVERR_SEQLENS
    assert torch.equal(got[0], good[0]) and bool((got[1] == 0).all())


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (256, 16, 2), (128, 12, 1)])
def test_nan_and_infinities_stay_where_they_are_seen(which, d, Hq, H):
    new = [1, 1, 1] if which == "decode" else [9, 3, 5]
    c = Case(61, new, [70, 30, 100], Hq, H, d, 16)
    clean = getattr(c, which)()
    rows = [slice(*c.cu.tolist()[b:b + 2]) for b in range(3)]
    G = Hq // H
    # a key with NaN: every row of its kv head that sees it
    c.cache[2][c.table[0, 1].long(), H - 1, 3, 0] = 255
    got = getattr(c, which)()
    assert bool(torch.isnan(got[rows[0], (H - 1) * G:]).all())
    assert torch.equal(got[rows[1]], clean[rows[1]]) and torch.equal(got[rows[2]], clean[rows[2]])
    assert torch.equal(got[rows[0], :(H - 1) * G], clean[rows[0], :(H - 1) * G])
    # a group of a value: its own 32 elements
    c.cache[3][c.table[1, 0].long(), 0, 5, 1] = 255
    got = getattr(c, which)()
    assert bool(torch.isnan(got[rows[1], :G, 32:64]).all())
    assert bool(torch.isfinite(got[rows[1], :G, :32]).all()) and bool(torch.isfinite(got[rows[1], G:]).all())
    assert torch.equal(got[rows[2]], clean[rows[2]])
    # a query that is not finite: its own head
    for bad in (torch.nan, torch.inf):
        q = c.q.clone()
        q[rows[2].start, 1, 7] = bad
        got = getattr(c, which)(q=q)
        assert bool(torch.isnan(got[rows[2].start, 1]).all())
        keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        keep[rows[2].start, 1] = False
        keep[rows[0]] = keep[rows[1]] = False
        assert torch.equal(got[keep], clean[keep])


# -------------------------------------------------------------------------------------- sizes of values

@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("spread", [12, 30])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (128, 8, 1), (256, 8, 1)])
def test_scales_far_apart(which, spread, d, Hq, H):
    """Groups of one token, and tokens of one block, whose scales differ by up to 2^spread."""
    new = [1, 1] if which == "decode" else [40, 70]
    c = Case(71 + spread, new, [300, 33], Hq, H, d, 32, spread=spread, q_size=3.0)
    c.check(getattr(c, which)(), which)


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_sharp_rows_and_growing_maxima(which):
    """Scores that grow along the keys by far more than the maximum may lag, and queries of 2^40."""
    new = [1] if which == "decode" else [3]
    c = Case(81, new, [900], 2, 1, 64, 64)
    n = int(c.lens[0])
    steps = torch.arange(c.W * 64, device="cuda").clamp(max=n) * 12 // n           # 2^0 .. 2^11
    for p in range(n):
        c.cache[2][c.table[0, p // 64].long(), 0, p % 64] = 118 + steps[p].to(torch.uint8)
    c.check(getattr(c, which)(), which)
    # V 2^60 times as large, queries 2^40 and keys 2^-40: the same rows, scaled (but for an exponent's rounding next to 60)
    c.cache[3] += 60
    c.cache[2] -= 40
    q = (c.q.double() * 2.0 ** 40).bfloat16()
    c.check(getattr(c, which)(q=q), which, q=q, v_exp=60)


def test_values_of_the_smallest_scales():
    """V's scales from 2^-90 on count in full; keys with far larger values next to them do not hide what a row sees."""
    c = Case(91, [1, 1], [199, 99], 4, 2, 64, 16)
    c.cache[3] -= 85
    c.check(c.decode(), "decode", v_exp=88)
    c.cache[3][c.table[0, 2].long(), :, 5] = 127 + 60
    c.check(c.decode(), "decode", v_exp=148)


# ------------------------------------------------------------------------------------------- prompts

@pytest.mark.parametrize("Hq,H,d,bs", [(2, 1, 64, 16), (16, 4, 64, 128), (7, 1, 128, 32), (16, 2, 128, 16), (16, 2, 256, 64), (3, 3, 256, 16)])
def test_prefill(Hq, H, d, bs):
    new = [1, 130, 17, 0, 64, 300]
    c = Case(Hq * 77 + d + bs, new, [0, 0, 33, 50, 128, 7], Hq, H, d, bs)
    got = c.prefill()
    c.check(got, "prefill")
    assert int(c.err) == 0
    assert torch.equal(c.prefill(held=c.blocks), got)          # (a request without new tokens needs no room)


def test_prefill_a_few_tokens_at_a_long_context():
    c = Case(7, [5, 1], [9000, 4000], 8, 2, 128, 64)
    c.check(c.prefill(), "prefill")


def test_prefill_rows_behind_the_last_sequence_and_refused_ones():
    """A padded step's rows stay as they were; a request whose keys are fewer than its tokens gives zeros for those that
    see nothing."""
    c = Case(8, [20, 9], [5, 30], 4, 2, 64, 16, slack=13)
    got = c.prefill()
    assert bool((got[c.T:] == 5.0).all())
    c.check(got[:c.T], "prefill", q=c.q[:c.T])
    c.lens[0] = 4          # the first 16 of its 20 tokens see nothing
    got = c.prefill()
    assert bool((got[:16] == 0).all()) and bool((got[16:c.T] != 0).any())
    c.check(got[:c.T], "prefill", q=c.q[:c.T])


def test_prefill_blocks_that_there_is_no_room_for():
    c = Case(9, [20, 30, 40], [100, 0, 60], 4, 2, 64, 16)     # 8, 2 and 7 blocks
    full = c.prefill()
    rows = c.cu.tolist()
    got = c.prefill(held=10)
    assert int(c.err) == gdn.GDN_DEVERR_BLOCKS | gdn.GDN_DEVERR_BLOCK_RANGE
    assert torch.equal(got[:rows[2]], full[:rows[2]]) and bool((got[rows[2]:] == 0).all())
    c.err.zero_()
    got = c.prefill(held=9)       # the second has no room, and no request behind one that has none
    assert int(c.err) == gdn.GDN_DEVERR_BLOCKS | gdn.GDN_DEVERR_BLOCK_RANGE
    assert torch.equal(got[:rows[1]], full[:rows[1]]) and bool((got[rows[1]:] == 0).all())


def test_prefill_lengths_that_are_none():
    c = Case(19, [4, 5, 6], [40, 40, 40], 4, 2, 64, 16)
    good = c.prefill()
    assert int(c.err) == 0
    rows = c.cu.tolist()
    c.lens[1], c.lens[2] = -3, c.W * 16 + 1
    got = c.prefill()
    assert int(c.err) & gdn.GDN_DEVERR_SEQLENS
    assert torch.equal(got[:rows[1]], good[:rows[1]]) and bool((got[rows[1]:rows[2]] == 0).all())


def test_prefill_more_requests_than_a_launch():
    """2,500 requests: two plans, one cache of pages."""
    new = [(i * 7) % 3 for i in range(2500)]
    c = Case(20, new, [(i * 13) % 40 for i in range(2500)], 2, 1, 64, 16)
    c.check(c.prefill(held=c.blocks), "prefill")
    assert int(c.err) == 0


def test_prefill_many_requests():
    """Requests by the hundred, some empty: their pages are counted by every CTA."""
    new = [(i * 7) % 5 for i in range(600)]
    c = Case(10, new, [(i * 13) % 60 for i in range(600)], 2, 1, 64, 16)
    got = c.prefill(held=c.blocks)
    c.check(got, "prefill")
    assert int(c.err) == 0


def test_prompts_do_not_depend_on_the_batch():
    new, old = [40, 130, 7], [100, 0, 500]
    c = Case(12, new, old, 8, 2, 128, 32)
    got, rows, table, lens, q = c.prefill(), c.cu.tolist(), c.table, c.lens, c.q
    for b in range(3):
        c.new, c.table, c.lens = [new[b]], table[b:b + 1].contiguous(), lens[b:b + 1].contiguous()
        c.cu = torch.tensor([0, new[b]], dtype=torch.int32, device="cuda")
        assert torch.equal(c.prefill(q=q[rows[b]:rows[b + 1]]), got[rows[b]:rows[b + 1]])


# ----------------------------------------------------------------------------- streams, graphs, together

def test_graphs_that_share_a_workspace():
    a, b = Case(13, [1] * 5, [300, 20, 700, 64, 1], 8, 2, 128, 32), Case(14, [40, 25], [10, 90], 8, 2, 128, 32)
    ws = torch.empty(max(gdn.gdn_attn4_decode_workspace_size(5, a.W, 8, 2, 128, 32), gdn.gdn_attn4_prefill_workspace_size(65, 2, b.W, 8, 2, 128, 32)),
                     dtype=torch.uint8, device="cuda")
    out_a, out_b = torch.empty_like(a.q), torch.empty_like(b.q)
    a.decode(out=out_a, ws=ws), b.prefill(out=out_b, ws=ws)
    graphs = []
    for f in (lambda: a.decode(out=out_a, ws=ws), lambda: b.prefill(out=out_b, ws=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    a.q.copy_(torch.randn_like(a.q, dtype=torch.float32))
    b.q.copy_(torch.randn_like(b.q, dtype=torch.float32))
    a.lens[0], a.lens[3] = 5, 0
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        out_a.zero_(), out_b.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        a.check(out_a, "decode")
        b.check(out_b, "prefill")


def test_two_calls_at_once():
    a, b = Case(15, [1] * 30, [500] * 30, 16, 2, 256, 64), Case(16, [200], [0], 16, 2, 256, 64)
    want_a, want_b = a.decode(), b.prefill()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            got_a = a.decode()
        with torch.cuda.stream(t):
            got_b = b.prefill()
        torch.cuda.synchronize()
        assert torch.equal(got_a, want_a) and torch.equal(got_b, want_b)


def test_no_requests():
    c = Case(17, [1], [3], 2, 1, 64, 16)
    q = c.q[:0]
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn4_decode(q, *c.cache, c.table[:0], c.lens[:0], torch.empty_like(q), ws)
    gdn.gdn_attn4_prefill(q, c.cu * 0, *c.cache, c.table, c.lens, torch.empty_like(q), ws)


def test_a_step_of_a_model():
    """Tables, positions, cache and attention as a server runs them: prompts, decode steps, speculation taken back. The
    cache's values are read back for the reference, so what is compared is the whole run."""
    Hq, H, d, bs, rot, NB = 8, 2, 128, 16, 64, 40
    new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = torch.int32
    cache = [new(NB, H, bs, d // 2, dtype=torch.uint8), new(NB, H, bs // 2, d, dtype=torch.uint8),
             new(NB, H, bs, d // 32, dtype=torch.uint8), new(NB, H, bs, d // 32, dtype=torch.uint8)]
    ring, pool, table, lens = torch.arange(NB, dtype=i, device="cuda"), torch.tensor([0, NB], dtype=i, device="cuda"), new(3, 12, dtype=i), new(3, dtype=i)
    err, rope = new(1, dtype=i), gdn.RopeTable(rot, base=1e6)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(0)
    kept = [(torch.empty(0, H, d), torch.empty(0, H, d)) for _ in range(3)]      # each request's keys (turned) and values
    for target in ([20, 3, 50], [21, 4, 51], [23, 4, 55], [22, 4, 52], [24, 5, 53], [1 + 24, 6, 54]):
        lens_new = torch.tensor(target, dtype=i, device="cuda")
        grown = [max(0, a - b) for a, b in zip(target, lens.tolist())]
        T = sum(grown) + 2                                                       # two rows of padding
        cu, slots, pos, before = new(4, dtype=i), new(T, dtype=i), new(T, dtype=i), lens.tolist()
        gdn.gdn_cache_tables(lens, lens_new, table, ring, pool, pool, cu, slots, pos, lens, bs, err=err)
        qkv = torch.randn(T, Hq + 2 * H, d, generator=gen).bfloat16().cuda()
        raw = qkv.clone()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        gdn.gdn_rope(q, k, pos, q, k, rope)
        gdn.gdn_cache4_append(k, v, slots, *cache, err=err)
        out = torch.full((T, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
        if all(g == 1 for g in grown):
            gdn.gdn_attn4_decode(q[:3], *cache, table, lens, out[:3], ws, err=err)
            which = "decode"
        else:
            gdn.gdn_attn4_prefill(q, cu, *cache, table, lens, out, ws, held_blocks=NB, err=err)
            which = "prefill"
        assert int(err) == 0 and lens.tolist() == target
        n = sum(grown)
        assert bool((out[n:] == 5.0).all()) and torch.equal(qkv[n:], raw[n:])     # padding
        for x, y in ((q, raw[:, :Hq]), (k, raw[:, Hq:Hq + H])):
            want, tol = co.rope(y[:n], pos[:n], rope.freqs, 1.0, rot, False)
            assert bool(((x[:n].double() - want).abs() <= tol).all())
        # what the cache holds is what was written, to half a step of each group
        kk, vv = co.unpack(*cache)
        for b in range(3):
            keep = min(before[b], target[b])
            rows = slice(*cu.tolist()[b:b + 2])
            kept[b] = tuple(torch.cat([old[:keep], x[rows].cpu().float()]) for old, x in zip(kept[b], (k, v)))
            at = torch.arange(target[b], device="cuda")
            for held, whole in zip(kept[b], (kk, vv)):
                got = whole[table[b, at // bs].long(), :, at % bs].cpu().unflatten(-1, (-1, 32))
                x = held.double().unflatten(-1, (-1, 32))
                assert bool(((got - x).abs() <= x.abs().amax(dim=-1, keepdim=True) * 2 / 7).all())
        want, tol = co.attention(q[:n], None if which == "decode" else cu.tolist(), kk, vv, table, lens, d ** -0.5, **ROUNDING[which](d))
        assert bool(((out[:n].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_a_large_cache(which):
    """Pages behind 2^32 bytes of a cache."""
    NB, H, bs, d = 70000, 4, 128, 256
    c = Case(18, [1, 1] if which == "decode" else [3, 30], [300, 200], 8, H, d, bs)
    n = c.cache[0].shape[0]
    big = [torch.zeros(NB, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in c.cache]
    assert big[0].numel() > 1 << 32
    for x, y in zip(big, c.cache):
        x[NB - n:] = y
    want = getattr(c, which)()
    c.check(want, which)
    c.cache = big
    c.table = torch.where(c.table >= 0, c.table + NB - n, -1).int()
    assert torch.equal(getattr(c, which)(), want) and int(c.err) == 0
