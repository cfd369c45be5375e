"""Calls of rotary positions that nothing else makes: keys alone, rows that do not start on 16 bytes, in and out of place by
different parts, one token with any strides."""
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


def rows(T, h, d, g, off=0, more=0):
    """[T, h, d] that starts `off` elements into its memory, `more` elements between tokens."""
    flat = torch.randn(T * (h * d + more) + off, generator=g).bfloat16().cuda()
    return flat[off:].view(T, h * d + more)[:, :h * d].unflatten(1, (h, d)), flat


@pytest.mark.parametrize("T", [1, 70])
def test_keys_alone(T):
    g = torch.Generator().manual_seed(T)
    k, _ = rows(T, 3, 64, g)
    pos, table = torch.arange(T, dtype=torch.int32, device="cuda") * 977, gdn.RopeTable(32)
    q, out = k[:, :0], torch.empty_like(k)
    gdn.gdn_rope(q, k, pos, q, out, table)
    check(out, k, pos, table, 32, False)


@pytest.mark.parametrize("T,h", [(1, 2), (9, 5), (300, 3)])
@pytest.mark.parametrize("off,more", [(1, 0), (4, 0), (8, 3), (0, 8), (0, 1)])
@pytest.mark.parametrize("which", ["in", "out", "both", "place"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_any_start_and_stride(T, h, off, more, which, interleaved):
    g = torch.Generator().manual_seed(T + off + more)
    x, flat = rows(T, h, 128, g, *((off, more) if which != "out" else (0, 0)))
    y, out = (x, flat) if which == "place" else rows(T, h, 128, g, *((off, more) if which != "in" else (0, 0)))
    before, was = x.clone(), out.clone()
    pos, table = torch.randint(0, 100000, (T,), generator=g).int().cuda(), gdn.RopeTable(64, base=5e5)
    gdn.gdn_rope(x, None, pos, y, None, table, interleaved=interleaved)
    check(y, before, pos, table, 64, interleaved)
    y.zero_()
    mask = out == 0                                      # what lies between and before the rows stays
    assert torch.equal(torch.where(mask, 0.0, was), torch.where(mask, 0.0, out))


def test_one_in_place_and_one_not():
    g = torch.Generator().manual_seed(5)
    q, k = rows(33, 4, 128, g)[0], rows(33, 2, 128, g)[0]
    pos, table = torch.arange(33, dtype=torch.int32, device="cuda"), gdn.RopeTable(48)
    for place_q in (True, False):
        a, b = q.clone(), k.clone()
        qo, ko = (a, torch.empty_like(b)) if place_q else (torch.empty_like(a), b)
        gdn.gdn_rope(a, b, pos, qo, ko, table)
        check(qo, q, pos, table, 48, False)
        check(ko, k, pos, table, 48, False)
