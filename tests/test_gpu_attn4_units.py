"""Single tokens over the 4-bit cache whose requests have more units than the join takes in one go: more than a
thread takes in order (16), and more than it keeps weights of at a time (1,024). How many units a length has is read off the workspace's size, so a
change of the rule that makes a request's units fewer fails here."""
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache4_oracle as co
from test_gpu_attn4 import Case

pytestmark = pytest.mark.gpu

UNIT = {64: 2048, 128: 2048, 256: 1024}     # keys of a long request's unit
IN_ORDER, WEIGHTS = 16, 1024


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def units(keys, Hq, H, d):
    """The most units that requests of up to `keys` keys have: each has (maximum, sum) and d sums in fp32 a head."""
    assert Hq == H or H == 1
    heads = Hq // H
    return gdn.gdn_attn4_decode_workspace_size(1, keys // 128, Hq, H, d, 128) // (H * heads * (8 + 4 * d))


@pytest.mark.parametrize("Hq,H,d", [(2, 1, 64), (9, 1, 128), (8, 1, 256)])
def test_more_units_than_one_thread_takes(Hq, H, d):
    n = (2 * IN_ORDER + 1) * UNIT[d]
    assert units(n, Hq, H, d) == 2 * IN_ORDER + 1
    lens = [x * UNIT[d] for x in (IN_ORDER, IN_ORDER + 1, 2 * IN_ORDER)] + [IN_ORDER * UNIT[d] + 1, n - 3, 5]
    c = Case(d + 1, [1] * len(lens), [x - 1 for x in lens], Hq, H, d, 128)
    c.check(c.decode(), "decode")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_more_units_than_weights_at_a_time(d):
    """1,026 units of pages that come again and again, but for the last two units, which have pages of their own with scores that
    make them about half of the sums."""
    unit, Hq = UNIT[d], 2
    most = WEIGHTS + 2
    n = most * unit
    assert units(n, Hq, 1, d) == most
    c = Case(d + 2, [1], [6 * unit - 1], Hq, 1, d, 128)
    c.q[:, 1] = (c.q[:, 0].double() * 0.875).bfloat16()
    each = unit // 128
    again, last = c.table[:, :4 * each], c.table[:, 4 * each:6 * each]
    # keys of the last two units: 6 with the query's signs (scores of about 7.2 and 6.3), next to 512 times as many about 0
    sign = torch.signbit(c.q[0, 0]).to(torch.uint8) * 8 + 7
    pages = last[0].long()
    c.cache[0][pages] = sign[0::2] | sign[1::2] << 4
    c.cache[2][pages] = 127
    c.table = torch.cat([again.repeat(1, WEIGHTS // 4), last], dim=1).contiguous()
    c.W = c.table.shape[1]
    assert c.W * 128 == n
    c.lens[:] = n - 5
    got = c.decode()
    k, v = co.unpack(*c.cache)
    pages = torch.cat([again[0], last[0]]).long()
    keys, vals = (x[pages, 0].reshape(-1, d) for x in (k, v))
    times = torch.ones(6 * unit, dtype=torch.float64, device="cuda")
    times[:4 * unit] = WEIGHTS // 4
    times[-5:] = 0
    s = c.q[0].double() @ keys.T * d ** -0.5
    p = torch.exp(s - s.amax(dim=1, keepdim=True)) * times
    share = p[:, 4 * unit:].sum(dim=1) / p.sum(dim=1)
    assert bool(((share > 0.05) & (share < 0.95)).all())
    want = p @ vals / p.sum(dim=1, keepdim=True)
    mag = p @ vals.abs() / p.sum(dim=1, keepdim=True)
    # probabilities to 11 bits; scores in fp32, twice (a key's and the maximum's): d terms, and an exponent of up to 40; sums
    # along a unit, then along every sixteenth unit, then of sixteen; the output to bf16
    score = d * 2.0 ** -23 * (c.q[0].double().abs().amax(dim=1, keepdim=True) * keys.abs().sum(dim=1).amax() * d ** -0.5) + 2.0 ** -18
    sums = (unit + most / 16 + 16) * 2.0 ** -23
    assert bool(((got[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * score + sums) * mag).all())
    assert int(c.err) == 0
