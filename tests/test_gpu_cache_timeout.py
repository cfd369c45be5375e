"""The bounded waits of the attention kernels running out, without faulting or hanging anything (include/gdn_testing.h): the
warp of CTA 0 that looks up pages leaves after four tiles, and the other roles' waits run out in turn, with copies and
products behind them. The call ends in bounded time with GDN_DEVERR_TIMEOUT in the error word, what the other CTAs computed is
what it always is, and so is the same call afterwards."""
import time

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


@pytest.fixture
def fault():
    yield gdn.gdn_testing_set_fault
    gdn.gdn_testing_set_fault(gdn.GDN_TEST_FAULT_NONE)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def cache(n_blocks, H, bs, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    pool = lambda: torch.randint(0, 120, (n_blocks, H, bs, d), device="cuda", generator=g, dtype=torch.uint8)  # noqa: E731
    return pool(), pool(), torch.full((n_blocks, H), 0.01, device="cuda"), torch.full((n_blocks, H), 0.01, device="cuda")


def broken_and_whole(call, fault, err):
    """The outputs of the call with the fault, and of the same call before and after."""
    whole = call().clone()
    assert int(err) == 0
    fault(gdn.GDN_TEST_FAULT_ATTENTION)
    t0 = time.monotonic()
    broken = call().clone()
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 20.0
    fault(gdn.GDN_TEST_FAULT_NONE)
    assert int(err) == gdn.GDN_DEVERR_TIMEOUT
    err.zero_()
    assert torch.equal(call(), whole) and int(err) == 0
    return broken, whole


@pytest.mark.parametrize("Hq,H,d", [(8, 2, 256), (8, 1, 128), (32, 2, 64)])
def test_decode(fault, Hq, H, d):
    B, n, bs = 40, 8000, 128                      # 40 H x 16 units over at most 304 CTAs: each has some
    kv = cache(63, H, bs, d)
    table = i32(list(range(63)))[None].expand(B, -1).contiguous()
    q = torch.randn(B, Hq, d, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    err = i32([0])
    ws = torch.empty(gdn.gdn_attn_decode_workspace_size(B, 63, Hq, H, d, bs), dtype=torch.uint8, device="cuda")

    def call():
        gdn.gdn_attn_decode(q, *kv, table, i32([n] * B), out, ws, err=err)
        return out

    broken, whole = broken_and_whole(call, fault, err)
    assert torch.equal(broken[B // 2:], whole[B // 2:])   # (CTA 0 has the first requests)


@pytest.mark.parametrize("Hq,H,d", [(8, 2, 256), (8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("old", [0, 9000])
def test_prefill(fault, Hq, H, d, old):
    T, bs = 900, 128
    W = -(-(old + T) // bs)
    kv = cache(W, H, bs, d)
    q = torch.randn(T, Hq, d, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    err = i32([0])
    ws = torch.empty(gdn.gdn_attn_prefill_workspace_size(T, 1, W, Hq, H, d, bs), dtype=torch.uint8, device="cuda")

    def call():
        gdn.gdn_attn_prefill(q, i32([0, T]), *kv, i32([list(range(W))]), i32([old + T]), out, ws, err=err)
        return out

    broken, whole = broken_and_whole(call, fault, err)
    # the (token, head) rows of one unit at most, or of the units that CTA 0 would have taken after it
    other = ((broken != whole) | broken.isnan()).any(dim=2).sum()
    assert int(other) <= 128 * 4
