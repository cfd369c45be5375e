"""Rotary positions on the GPU against the 64-bit restatement of tests/_cache4_oracle.py."""
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


def check(got, x, pos, table, rot, interleaved):
    want, tol = co.rope(x, pos, table.freqs, table.factor, rot, interleaved)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert torch.equal(got[..., rot:], x[..., rot:])            # copied as it is


# (T, Hq, Hkv, d, rot): vectors and single elements, one token to many, odd numbers of heads, all of a head to two elements
SIZES = [(1, 16, 2, 256, 64), (5, 1, 1, 64, 64), (64, 28, 4, 128, 128), (1500, 3, 1, 96, 48), (7, 5, 2, 80, 80), (3, 2, 2, 80, 20),
         (9, 4, 1, 6, 2), (2, 1, 1, 5, 4), (1030, 2, 1, 64, 2), (33, 7, 3, 1024, 1024), (4, 3, 1, 128, 126), (2, 1, 1, 16, 16),
         (3, 1, 0, 48, 16), (1025, 1, 0, 16, 16)]


@pytest.mark.parametrize("T,Hq,H,d,rot", SIZES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, Hq, H, d, rot, interleaved):
    g = torch.Generator().manual_seed(T * 7 + d + rot)
    qkv = torch.randn(T, Hq + 2 * H + 1, d, generator=g).bfloat16().cuda()        # slices of one projection
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + H]
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int().cuda()
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 1 << 24, 0x7fffffff
    table = gdn.RopeTable(rot, base=5e5, scaling="linear" if T % 2 else "none", factor=1.5)
    q_out, k_out = torch.full_like(qkv[:, :Hq + 1], 9.0)[:, :Hq], torch.full((T, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_rope(q, k if H else None, pos, q_out, k_out if H else None, table, interleaved=interleaved)
    # at 2^31 a table from doubles is off by 2^-53 / (2 pi) * 2^31 of a turn: 2^-24
    far = pos > 1 << 24
    for got, x in ((q_out, q), (k_out, k)):
        want, tol = co.rope(x, pos, table.freqs, table.factor, rot, interleaved)
        size = x.double().abs().amax(dim=-1, keepdim=True) * table.factor * 2 * 2.0 ** -20
        assert bool(((got.double() - want).abs() <= tol + torch.where(far[:, None, None], size, 0.0)).all())
        assert torch.equal(got[..., rot:], x[..., rot:])
    # in place, and the projection's other elements as they were
    other = qkv[:, Hq + H:].clone()
    gdn.gdn_rope(q, k if H else None, pos, q, k if H else None, table, interleaved=interleaved)
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(qkv[:, Hq + H:], other)


@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)])
def test_scaled_for_long_contexts(scaling, factor):
    table = gdn.RopeTable(128, base=1e6, scaling=scaling, factor=factor, trained_len=32768)
    q = torch.randn(300, 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    pos = torch.arange(500_000, 500_300, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    gdn.gdn_rope(q, None, pos, out, None, table)
    check(out, q, pos, table, 128, False)
    assert (table.factor > 1) == (scaling == "yarn")


def test_a_models_own_frequencies():
    w = [1.0, 0.5, 0.1, 3.0, 0.0, -0.25, 1e-3, 7.0]
    table = gdn.RopeTable(16, freqs=w, factor=0.75)
    q = torch.randn(40, 3, 32).bfloat16().cuda()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    gdn.gdn_rope(q, None, pos, out, None, table, interleaved=True)
    check(out, q, pos, table, 16, True)


@pytest.mark.parametrize("d,rot", [(128, 64), (30, 10)])
def test_padding_and_values_that_are_not_finite(d, rot):
    """Negative positions leave their rows alone; NaN and infinities reach their own pair, the rest of a head is copied."""
    q = torch.randn(9, 2, d).bfloat16().cuda()
    q[2, 0, 1], q[3, 1, rot - 1], q[4, 0, d - 1] = torch.nan, torch.inf, torch.nan
    pos = torch.tensor([5, -1, 7, 9, 11, -1, 13, -5, -1], dtype=torch.int32, device="cuda")
    table = gdn.RopeTable(rot)
    out = torch.full_like(q, 3.0)
    gdn.gdn_rope(q, None, pos, out, None, table)
    assert bool((out[pos < 0] == 3.0).all())
    live = pos >= 0
    want, tol = co.rope(q, pos, table.freqs, 1.0, rot, False)
    finite = torch.isfinite(want) & torch.isfinite(tol)
    assert bool((((out.double() - want).abs() <= tol) | ~finite)[live].all())
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[2, 0, 1], [2, 0, 1 + rot // 2], [3, 1, rot // 2 - 1], [3, 1, rot - 1], [4, 0, d - 1]]


def test_a_row_alone_and_in_a_batch_on_streams_and_in_graphs():
    table = gdn.RopeTable(64, base=1e7)
    q = torch.randn(2000, 4, 128).bfloat16().cuda()
    pos = torch.randint(0, 100000, (2000,), dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    gdn.gdn_rope(q, None, pos, out, None, table)
    for t in (0, 7, 1999):
        one = torch.empty_like(q[t:t + 1])
        gdn.gdn_rope(q[t:t + 1], None, pos[t:t + 1], one, None, table)
        assert torch.equal(one, out[t:t + 1])
    side = torch.cuda.Stream()
    got = torch.empty_like(q)
    torch.cuda.synchronize()
    gdn.gdn_rope(q, None, pos, got, None, table, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    again = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_rope(q, None, pos, again, None, table)
    q.copy_(torch.randn_like(q, dtype=torch.float32))
    gdn.gdn_rope(q, None, pos, out, None, table)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    gdn.gdn_rope(q[:0], None, pos[:0], out[:0], None, table)      # nothing to do
