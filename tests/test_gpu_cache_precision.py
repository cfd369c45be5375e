"""What attention over the 8-bit cache keeps of a softmax that is not flat: one key far above the others, blocks of
values whose scales differ by many powers of two, values that a row does not see. Against plain 64-bit attention,
element by element, within what the kernels say they round (include/gdn.h): a probability to `bits` significant bits
and to `floor` of the row's largest probability x scale of V, a query to 2^-18 of its row's largest element, sums in
fp32, the result to bf16."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache_oracle as co

pytestmark = pytest.mark.gpu

# (significant bits, floor) of a probability
KEEPS = {("prefill", 64): (11, 2.0 ** -32), ("prefill", 128): (11, 2.0 ** -32), ("prefill", 256): (11, 2.0 ** -28),
         ("decode", 64): (16, 2.0 ** -26), ("decode", 128): (16, 2.0 ** -26), ("decode", 256): (16, 2.0 ** -26)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pages:
    """A cache of the given keys and values [n, H, d] of one request, in shuffled pages; the bytes and scales of a page
    by its largest element."""

    def __init__(self, k, v, bs, seed=0):
        n, self.H, self.d = k.shape
        self.n, self.bs, W = n, bs, -(-n // bs)
        perm = torch.from_numpy(np.random.default_rng(seed).permutation(W + 2)).cuda()
        self.table = perm[:W].to(torch.int32)[None].contiguous()

        def pool(x):
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, W * bs - n)).view(W, bs, self.H, self.d).transpose(1, 2)
            s = (x.abs().amax(dim=(2, 3)) / 448).clamp(min=2.0 ** -64)
            c = torch.full((W + 2, self.H, bs, self.d), 0x7F, dtype=torch.uint8, device="cuda")  # (NaN where no page is)
            c[self.table[0].long()] = (x / s[:, :, None, None]).clamp(-448, 448).to(co.F8).view(torch.uint8)
            all_s = torch.ones(W + 2, self.H, device="cuda")
            all_s[self.table[0].long()] = s
            return c, all_s

        (self.kc, self.ks), (self.vc, self.vs) = pool(k), pool(v)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def pools(self):
        return self.kc, self.vc, self.ks, self.vs

    def values(self, cache, scale):
        lut = torch.from_numpy(co.E4M3).cuda()
        p = self.table[0].long()
        x = lut[cache[p].long()] * scale[p].double()[:, :, None, None]
        return x.transpose(1, 2).reshape(-1, self.H, self.d)[:self.n]

    def scale_of(self, scale):  # of each key's page, [n, H]
        return scale[self.table[0].long()].double().repeat_interleave(self.bs, 0)[:self.n]


def run(c, q, which):
    """The rows of q as the last tokens of the request; `decode`: each by itself, as a batch."""
    T, Hq, d = q.shape
    out = torch.full_like(q, 7.0)
    if which == "decode":
        table = c.table.expand(T, -1).contiguous()
        lens = i32(np.arange(c.n - T + 1, c.n + 1))
        ws = torch.empty(gdn.gdn_attn_decode_workspace_size(T, table.shape[1], Hq, c.H, d, c.bs), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_decode(q, *c.pools(), table, lens, out, ws, err=c.err)
    else:
        ws = torch.empty(gdn.gdn_attn_prefill_workspace_size(T, 1, c.table.shape[1], Hq, c.H, d, c.bs), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_prefill(q, i32([0, T]), *c.pools(), c.table, i32([c.n]), out, ws, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    return out


def exact(c, q, which):
    """The result in 64 bits and the bound: see the head of this file."""
    T, Hq, d = q.shape
    G = Hq // c.H
    bits, floor = KEEPS[which, d]
    k, v = c.values(c.kc, c.ks), c.values(c.vc, c.vs)
    vs = c.scale_of(c.vs)
    hidden = torch.arange(c.n, device="cuda")[None, :] > (c.n - T + torch.arange(T, device="cuda"))[:, None]
    out = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda")
    tol = torch.empty_like(out)
    for m in range(Hq):
        h = m // G
        x = q[:, m].double()
        s = (x @ k[:, h].T * d ** -0.5).masked_fill(hidden, -torch.inf)
        p = torch.softmax(s, dim=1)
        vh = torch.where(v[:, h].isnan(), 0.0, v[:, h])
        o = p @ vh
        out[:, m] = o
        # a score: queries 2^-18 of the largest element, fp32 sums over d; twice for the key and for the maximum
        size = x.abs().amax(dim=1, keepdim=True) * k[:, h].abs().sum(dim=1).amax() * d ** -0.5
        e = 2 * ((2.0 ** -18 + d * 2.0 ** -24) * size + 2.0 ** -21 * (1 + torch.where(hidden, 0.0, s).abs().amax(dim=1, keepdim=True)))
        mag = p @ vh.abs()
        least = (p * vs[:, h]).amax(dim=1, keepdim=True) * floor * ((~hidden).double() @ (vh.abs() / vs[:, h, None]).nan_to_num())
        tol[:, m] = (2.0 ** -bits + e + c.n * 2.0 ** -24) * mag + least + 2.0 ** -8 * o.abs() + 1e-38
    return out, tol


def check(c, q, which):
    want, tol = exact(c, q, which)
    got = run(c, q, which).double()
    assert bool(torch.isfinite(got).all())
    off = (got - want).abs()
    assert bool((off <= tol).all()), (float((off / tol).max()), float((off.norm() / want.norm())))


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, device="cuda", generator=g)


def one_key_above(which, T, Hq, H, d, gap, flat, n=5003):
    """The usual first token: `gap` nats above the rest, a value of next to nothing, so that what comes out is the sum of
    many small probabilities; with `flat` they are all the same and their rounding does not average out."""
    r = rand(gap + d)
    u = torch.sign(r(d)) * 0.5
    k = (0.0 if flat else 0.6) * r(n, H, d)
    k[0] = u * (gap / (0.25 * d ** 0.5))
    v = 1.0 + 0.3 * r(n, H, d)
    v[0] = 0.002
    q = (u + (0.0 if flat else 0.05) * r(T, Hq, d)).bfloat16()
    check(Pages(k, v, 16, gap), q, which)


def one_key_above_a_long_request(which, T, d):
    n, r = 60000, rand(d)
    u = torch.sign(r(d)) * 0.5
    k = 0.4 * r(n, 1, d)
    k[0] = u * (11 / (0.25 * d ** 0.5))
    v = 1.0 + r(n, 1, d)
    v[0] = 0.01
    check(Pages(k, v, 64), (u + 0.05 * r(T, 4, d)).bfloat16(), which)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("Hq,H", [(4, 2), (16, 2)])
@pytest.mark.parametrize("gap", [6, 10, 12, 16])
@pytest.mark.parametrize("flat", [False, True])
def test_prompts_256_one_key_above_the_others(T, Hq, H, gap, flat):
    one_key_above("prefill", T, Hq, H, 256, gap, flat)


def test_prompts_256_one_key_above_a_long_request():
    one_key_above_a_long_request("prefill", 70, 256)


HEADS = [(4, 2, 64), (16, 2, 64), (8, 2, 128), (16, 1, 128), (4, 2, 256), (16, 2, 256)]


@pytest.mark.parametrize("which,T", [("decode", 3), ("prefill", 5), ("prefill", 300)])
@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("power", [-20, 14, 30])
def test_a_block_of_other_values_that_has_no_weight(which, T, Hq, H, d, power):
    """A page whose values are 2^power times the others', 50 nats below them: it decides nothing."""
    n, r = 2100, rand(power + 100)
    u = torch.sign(r(d)) * 0.5
    k, v = 0.5 * r(n, H, d), 1.0 + r(n, H, d)
    k[640:656] -= u * (50 / (0.25 * d ** 0.5))
    v[640:656] *= 2.0 ** power
    check(Pages(k, v, 16), (u + 0.05 * r(T, Hq, d)).bfloat16(), which)


@pytest.mark.parametrize("which,T", [("decode", 3), ("prefill", 5), ("prefill", 300)])
@pytest.mark.parametrize("Hq,H,d", HEADS)
def test_weight_on_a_block_of_small_values(which, T, Hq, H, d):
    """The other way round: most of the probability on a page whose values are 2^-18 of the others'."""
    n, r = 1500, rand(d)
    u = torch.sign(r(d)) * 0.5
    k, v = 0.5 * r(n, H, d), 1.0 + r(n, H, d)
    k[320:336] += u * (9 / (0.25 * d ** 0.5))
    v[320:336] *= 2.0 ** -18
    check(Pages(k, v, 16), (u + 0.05 * r(T, Hq, d)).bfloat16(), which)


@pytest.mark.parametrize("which,T", [("decode", 1), ("prefill", 40)])
@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("power", [0, -40, 100])
def test_blocks_of_zeros(which, T, Hq, H, d, power):
    """Pages of zeros, whose scale is the writer's least (2^-64), and some of scale 0, between pages of any size: their
    keys count in the sum."""
    n, r = 700, rand(power + d)
    k, v = r(n, H, d), (1.0 + r(n, H, d)) * 2.0 ** power
    v[0:64] = v[200:300] = v[500:560] = 0.0
    c = Pages(k, v, 16)
    c.vs[c.table[0, 14:16].long()] = 0.0
    check(c, r(T, Hq, d).bfloat16(), which)


@pytest.mark.parametrize("Hq,H,d", [(4, 2, 64), (8, 2, 128), (16, 2, 256)])
@pytest.mark.parametrize("old", [0, 100, 5000])
def test_later_tokens_of_any_size(Hq, H, d, old):
    """What a row does not see: tokens after it, their pages' scales of any size."""
    T, r = 200, rand(old + d)
    k, v = r(old + T, H, d), 1.0 + r(old + T, H, d)
    first = -(-(old + 90) // 16) * 16
    v[first:] *= 2.0 ** 25
    check(Pages(k, v, 16), r(T, Hq, d).bfloat16(), "prefill")


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("Hq,H,d", HEADS[:4])
@pytest.mark.parametrize("gap", [6, 10, 16, 18])
@pytest.mark.parametrize("flat", [False, True])
def test_prompts_64_128_one_key_above_the_others(T, Hq, H, d, gap, flat):
    one_key_above("prefill", T, Hq, H, d, gap, flat)


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("gap", [6, 10, 14, 16])
@pytest.mark.parametrize("flat", [False, True])
def test_single_tokens_one_key_above_the_others(Hq, H, d, gap, flat):
    one_key_above("decode", 3, Hq, H, d, gap, flat)
    one_key_above("decode", 3, Hq, H, d, gap, flat, n=250)   # (all that is looked at together)


@pytest.mark.parametrize("which,T,d", [("decode", 2, 64), ("decode", 2, 128), ("decode", 2, 256), ("prefill", 70, 64), ("prefill", 70, 128)])
def test_one_key_above_a_long_request(which, T, d):
    one_key_above_a_long_request(which, T, d)


@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("old,T", [(0, 5), (0, 300), (90, 129), (5000, 64), (20000, 40)])
def test_nan_in_a_value_stays_with_the_rows_that_see_it(Hq, H, d, old, T):
    """NaN among the values of tokens, a column or all of them: in the columns of the rows that see it, and nowhere else;
    NaN keys of tokens that a row does not see do nothing."""
    n, r = old + T, rand(old + T + d)
    c = Pages(r(n, H, d), r(n, H, d), 16)
    q = r(T, Hq, d).bfloat16()
    put = [(n - 1, 0, slice(None)), (n - 1 - T // 2, H - 1, slice(3, 4)), (old + T // 4, 0, slice(d - 1, d)), (old, H - 1, slice(17, 20))]
    if old:
        put.append((old // 2, 0, slice(5, 6)))
    at = lambda pos: (int(c.table[0, pos // 16]), pos % 16)  # noqa: E731
    for pos, h, cols in put:
        c.vc[at(pos)[0], h, at(pos)[1], cols] = 0
    want = run(c, q, "prefill").clone()
    for pos, h, cols in put:
        c.vc[at(pos)[0], h, at(pos)[1], cols] = 0xFF if pos % 2 else 0x7F
        want[max(pos - old, 0):, h * (Hq // H):(h + 1) * (Hq // H), cols] = float("nan")
    got = run(c, q, "prefill")
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())

    if T > 8:  # keys
        c.kc[at(n - 3)[0], :, at(n - 3)[1]] = 0x7F
        got = run(c, q, "prefill")
        assert torch.equal(got[:-3].isnan(), want[:-3].isnan()) and torch.equal(got[:-3].nan_to_num(), want[:-3].nan_to_num())
        assert bool(got[-3:].isnan().all())


@pytest.mark.parametrize("Hq,H,d", [(4, 2, 64), (8, 2, 128), (16, 2, 256)])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -1.0, 0.0, 3e38, 1e-45])
def test_scales_of_pages_that_a_row_does_not_see(Hq, H, d, scale):
    """Whatever stands for the scales of later tokens' pages: the rows before them do not change."""
    old, T = 100, 60
    n, r = old + T, rand(d)
    c = Pages(r(n, H, d), r(n, H, d), 16)
    q = r(T, Hq, d).bfloat16()
    want = run(c, q, "prefill")[:28].clone()
    for which in (c.vs, c.ks):
        page = c.table[0, 8:].long()          # tokens 128 on: row 28 is the first to see one
        was = which[page].clone()
        which[page] = scale
        assert torch.equal(run(c, q, "prefill")[:28], want)
        which[page] = was


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_one_token_of_any_stride(which):
    """The stride of a single token is not used: torch gives any."""
    n, H, Hq, d, r = 40, 2, 4, 64, rand(1)
    c = Pages(r(n, H, d), r(n, H, d), 16)
    q = r(1, Hq, d).bfloat16()
    for step in (0, 1, Hq * d + 4, 10 ** 6 + 1):
        want = run(c, q, which)  # (the writes below change a page's scale)
        odd = q.as_strided(q.shape, (step, d, 1))
        out = torch.empty(1, Hq, d, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        if which == "decode":
            gdn.gdn_attn_decode(odd, *c.pools(), c.table, i32([n]), out, ws)
        else:
            gdn.gdn_attn_prefill(odd, i32([0, 1]), *c.pools(), c.table, i32([n]), out, ws)
        assert torch.equal(out, want)
        k = r(1, H, d).bfloat16()
        odd = k.as_strided(k.shape, (step, d, 1))
        gdn.gdn_cache_append(odd, odd, i32([int(c.table[0, 2]) * 16 + 9]), *c.pools())
        kept = run(c, q, which)
        gdn.gdn_cache_append(k, k, i32([int(c.table[0, 2]) * 16 + 9]), *c.pools())
        assert torch.equal(run(c, q, which), kept)


@pytest.mark.parametrize("which,T", [("decode", 2), ("prefill", 3), ("prefill", 200)])
@pytest.mark.parametrize("Hq,H,d", HEADS)
@pytest.mark.parametrize("power", [-78, -50, 60, 100])
def test_values_of_any_size(which, T, Hq, H, d, power):
    """All values of a request as small as scales of 2^-90, and as large as bf16 has room for."""
    n, r = 1000, rand(power + 200)
    c = Pages(r(n, H, d), 1.0 + r(n, H, d), 16)
    c.vs *= 2.0 ** power
    check(c, r(T, Hq, d).bfloat16(), which)
