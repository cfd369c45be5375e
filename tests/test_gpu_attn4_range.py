"""Attention over the 4-bit cache near the ends of what its scales can say, against the 64-bit restatement of
tests/_cache4_oracle.py: scales of K next to 2^127, queries next to 2^-120,
values below 2^-90 and
next to 2^127."""
import pytest
import torch

import _cache4_oracle as co
import test_gpu_cache_precision as eight
from test_gpu_attn4 import ROUNDING, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("up", [64, 68, 100, 112])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (128, 9, 1), (256, 16, 2)])
def test_large_keys(which, up, d, Hq, H):
    """Keys 2^up times as large (bytes up to 127 + up) and queries as much smaller: the scores are the usual ones. Then every
    third key as it was: its scores are 0 to 2^-60, next to the others' in the same tiles."""
    new = [1, 1] if which == "decode" else [9, 40]
    c = Case(101 + up, new, [300, 33], Hq, H, d, 32, q_size=3.0)
    # (elements of 2^-120 and less have 8 bits in bf16, those below 2^-126 fewer: the reference takes what is there)
    q = (c.q.double() * 2.0 ** -up).bfloat16()
    c.cache[2] += up
    got = getattr(c, which)(q=q)
    assert bool(torch.isfinite(got).all())
    c.check(got, which, q=q)
    c.cache[2][:, :, ::3] -= up
    c.check(getattr(c, which)(q=q), which, q=q)
    assert int(c.err) == 0


def test_a_large_key_that_no_one_sees():
    """Scales of 2^127 behind the last token of a request and in other heads change no bit of its rows."""
    c = Case(7, [1], [40], 4, 2, 64, 16)
    clean = c.decode()
    c.cache[2][c.table[0, 2].long(), :, 9:] = 254        # (41 tokens: the third page has nine)
    assert torch.equal(c.decode(), clean)
    c.cache[2][c.table[0, 2].long(), 1] = 254
    assert torch.equal(c.decode()[:, :2], clean[:, :2])


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("up", [116, 119, 122])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (128, 9, 1), (256, 16, 2)])
def test_small_queries(which, up, d, Hq, H):
    """Queries whose largest element is around 2^-120, with keys as much larger."""
    c = Case(131 + up, [1, 1] if which == "decode" else [9, 40], [300, 33], Hq, H, d, 32, q_size=3.0)
    q = (c.q.double() * 2.0 ** -up).bfloat16()
    c.cache[2] += up
    c.check(getattr(c, which)(q=q), which, q=q)


@pytest.mark.parametrize("which,T", [("decode", 5), ("prefill", 300)])
@pytest.mark.parametrize("up", [112, 118, 121])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_small_queries_over_the_8_bit_cache(which, T, up, d):
    r = eight.rand(up + d)
    k, v = r(700, 2, d) * 2.0 ** up, 1.0 + 0.3 * r(700, 2, d)
    q = (r(T, 8, d).double() * 2.0 ** -up).bfloat16()
    eight.check(eight.Pages(k, v, 16), q, which)


@pytest.mark.parametrize("down", [60, 80, 86, 92, 100, 115])
@pytest.mark.parametrize("d,Hq,H", [(64, 4, 2), (128, 9, 1), (256, 16, 2)])
def test_small_values_of_prompts(down, d, Hq, H):
    """Values of 2^-60 to 2^-115: exact in a block's 8 bits as long as its largest scale is 2^-84 or more, in steps of 2^-99 below
    that (half a step for each value, and so for their mean)."""
    c = Case(151 + down, [9, 40], [300, 33], Hq, H, d, 32)
    c.cache[3] -= down
    got = c.prefill()
    k, v = co.unpack(*c.cache)
    want, tol = co.attention(c.q, c.cu.tolist(), k, v, c.table, c.lens, d ** -0.5, v_exp=down + 3, **ROUNDING["prefill"](d))
    # (the restatement's bound ends in 1e-30, which is larger than some of these values)
    tol = tol - 0.999 * 1e-30 + (1.01 * 2.0 ** -100 if down > 80 else 0)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("up", [60, 100, 112, 119, 125])
@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 16), (256, 3)])
def test_a_large_value_among_many_small_ones(up, d, Hq):
    """One key with nearly all of a row's largest probability and a value of 2^up, 70,000 with 2^-17 of it each: together they
    are a third of the sum."""
    n, bs = 70001, 64
    c = Case(171 + up, [1], [n - 1], Hq, 1, d, bs)
    c.q = torch.where(c.q > 0, 0.5, -0.5).bfloat16()
    c.cache[0].zero_()
    c.cache[2][:] = 127
    at = 30000                                            # the key: k with the queries' signs (the heads have the same)
    c.q[:] = c.q[:, :1]
    score = 0.5 * d * d ** -0.5                           # ... of a key of ones
    k = {64: 3.0, 128: 2.0, 256: 1.5}[d]                  # exact codes; 12, 11.3 and 12 nats
    code = {3.0: 5, 2.0: 4, 1.5: 3}[k]
    assert 11 < score * k < 12.5
    sign = torch.signbit(c.q[0, 0]).to(torch.uint8) * 8 + code
    c.cache[0][c.table[0, at // bs].long(), 0, at % bs] = sign[0::2] | sign[1::2] << 4
    c.cache[3][c.table[0, at // bs].long(), 0, at % bs] = 127 + up
    c.cache[1][c.table[0, at // bs].long(), 0, at % bs // 2] = 0x21       # 0.5 (the even token, 30,000) and 1
    got = c.decode()
    c.check(got, "decode", v_exp=up)


@pytest.mark.parametrize("up", [100, 123, 125, 126])
@pytest.mark.parametrize("d,Hq,k", [(64, 2, 2.0), (128, 16, 1.5), (256, 3, 1.0)])
def test_a_large_value_in_a_unit(up, d, Hq, k):
    """The same within one unit (256, 512 or 1,024 keys): one key of 2^up next to keys with 2^-11.5 or 2^-12.2 of its probability,
    where a sum that ends at 2^-126 is off by a tenth to a third from 2^124 or 2^123 on."""
    n, bs, at = {64: 1024, 128: 512, 256: 256}[d], 32, 100
    c = Case(191 + up, [1], [n - 1], Hq, 1, d, bs)
    c.q[:] = torch.where(c.q[:, :1] > 0, 0.5, -0.5)
    c.cache[0].zero_()
    c.cache[2][:] = 127
    page = c.table[0, at // bs].long()
    sign = torch.signbit(c.q[0, 0]).to(torch.uint8) * 8 + {2.0: 4, 1.5: 3, 1.0: 2}[k]
    c.cache[0][page, 0, at % bs] = sign[0::2] | sign[1::2] << 4
    c.cache[3][page, 0, at % bs] = 127 + up
    c.cache[1][page, 0, at % bs // 2] = 0x21              # the (even) token's values are 0.5 * 2^up
    got = c.decode()
    c.check(got, "decode", v_exp=up)
    share = n * 2.0 ** (-k * 0.5 * d ** 0.5 * 1.4427)
    assert share > 0.08 and bool((got.double() < 2.0 ** (up - 1) / (1 + 0.9 * share)).all())


@pytest.mark.parametrize("which,T,up", [("decode", 3, 108), ("prefill", 40, 72)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_large_value_over_the_8_bit_cache(which, T, up, d):
    """What the header says of a row's sum: with a v_scale of up to 2^100 (prompts 2^64) it has what is far below its largest.
    One value of 2^up, 1,500 keys with about 2^-12 of its probability."""
    r = eight.rand(d)
    u = torch.sign(r(d)) * 0.5
    k = 0.2 * r(1500, 1, d)
    k[0] = u * (8 / (0.25 * d ** 0.5))
    v = 1.0 + 0.3 * r(1500, 1, d)
    v[0] = 2.0 ** up * (1.0 + 0.3 * r(d).clamp(-2, 2))
    q = (u + 0.02 * r(T, 4, d)).bfloat16()
    c = eight.Pages(k, v, 16)
    assert up - 9 < float(torch.log2(c.vs.max())) < up - 8 + 0.1
    eight.check(c, q, which)


@pytest.mark.parametrize("d,k", [(64, 2.0), (128, 1.5), (256, 1.0)])
def test_a_large_value_in_prompts(d, k):
    """The same over the 4-bit cache: a group's scale of 2^70 is a block's of 2^64."""
    n, bs, at = 1024, 32, 100
    c = Case(211, [9], [n - 9], 2, 1, d, bs)
    c.q[:] = torch.where(c.q[:1, :1] > 0, 0.5, -0.5)
    c.cache[0].zero_()
    c.cache[2][:] = 127
    page = c.table[0, at // bs].long()
    sign = torch.signbit(c.q[0, 0]).to(torch.uint8) * 8 + {2.0: 4, 1.5: 3, 1.0: 2}[k]
    c.cache[0][page, 0, at % bs] = sign[0::2] | sign[1::2] << 4
    c.cache[3][page, 0, at % bs] = 127 + 70
    c.check(c.prefill(), "prefill", v_exp=70)
