"""Rotary positions around the counts of tokens at which a token gets fewer threads: the rows of a call are those of one token at
a time, bit for bit."""
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

from test_gpu_rope import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("T", [256, 257, 1024, 1025])
@pytest.mark.parametrize("Hq,H,d,rot", [(5, 2, 128, 128), (3, 1, 1024, 1024), (130, 1, 64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_threads(T, Hq, H, d, rot, interleaved):
    g = torch.Generator().manual_seed(T + d)
    q, k = torch.randn(T, Hq, d, generator=g).bfloat16().cuda(), torch.randn(T, H, d, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int().cuda()
    pos[3] = -1
    table = gdn.RopeTable(rot, base=1e6)
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    gdn.gdn_rope(q, k, pos, q_out, k_out, table, interleaved=interleaved)
    assert bool((q_out[3] == 7.0).all()) and bool((k_out[3] == 7.0).all())
    live = pos >= 0
    check(q_out[live], q[live], pos[live], table, rot, interleaved)
    check(k_out[live], k[live], pos[live], table, rot, interleaved)
    for t in (0, T // 2, T - 1):
        a, b = torch.empty_like(q[:1]), torch.empty_like(k[:1])
        gdn.gdn_rope(q[t:t + 1], k[t:t + 1], pos[t:t + 1], a, b, table, interleaved=interleaved)
        assert torch.equal(a[0], q_out[t]) and torch.equal(b[0], k_out[t])
    gdn.gdn_rope(q, k, pos, q, k, table, interleaved=interleaved)
    assert torch.equal(q[live], q_out[live]) and torch.equal(k[live], k_out[live])
