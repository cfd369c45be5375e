"""Sizes at the top of what 32-bit indices hold, through the C ABI, without a GPU: refused before any CUDA call, or split
into launches that stay below (seen in the workspace's size)."""
import ctypes
import os
import re

import pytest

import gated_deltanet_linear_gdn_gb300 as gdn
from gated_deltanet_linear_gdn_gb300 import build

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its checks first
INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return gdn.lib()


def decode(L, B, W, q, kv, d=64, bs=128, size=1 << 62):
    dims = gdn.gdn_cache_dims(q, kv, d, bs)
    return L.gdn_attn_decode(FAKE, 1024 * d, FAKE, FAKE, FAKE, FAKE, 10, FAKE, W, FAKE, B, dims, 0.1, FAKE, FAKE, size, None, None)


def test_decode_tiles_of_a_launch(L):
    """Tiles of 128 keys x kv heads x groups of 16 query heads, over a launch's requests, are counted in 32 bits."""
    size = gdn.gdn_attn_decode_workspace_size
    # one request of 2^24 blocks of 128 for 1,024 kv heads: 2^34 tiles
    assert decode(L, 1, (1 << 24) - 20, 1024, 1024) == UNS and size(1, (1 << 24) - 20, 1024, 1024, 64, 128) == 0
    # 2^21 tiles a head: 1,023 fit, and 1,024 don't
    assert decode(L, 1, 1 << 21, 1024, 1024) == UNS
    assert decode(L, 1, 1 << 21, 1023, 1023, size=100) == INV        # (supported: the workspace is too small)
    # 2^16 tiles, 128 heads: 2^23 a request, 255 of them in a launch
    assert size(255, 1 << 16, 128, 128, 64, 128) == size(256, 1 << 16, 128, 128, 64, 128) == size(9999, 1 << 16, 128, 128, 64, 128)
    assert size(254, 1 << 16, 128, 128, 64, 128) < size(255, 1 << 16, 128, 128, 64, 128)
    # ordinary sizes take as many requests a launch as before
    assert size(319, 1 << 10, 32, 8, 128, 64) < size(320, 1 << 10, 32, 8, 128, 64) == size(321, 1 << 10, 32, 8, 128, 64)


def tables(L, T, W=4, bs=16):
    return L.gdn_cache_tables(FAKE, FAKE, 3, FAKE, W, FAKE, 20, FAKE, FAKE, bs, T, FAKE, FAKE, P(0x10001), FAKE, None, None)


def append(L, T, N=10, kv=1):
    return L.gdn_cache_append(FAKE, 64 * kv, P(0x10002), 64 * kv, FAKE, T, FAKE, FAKE, FAKE, FAKE, N, gdn.gdn_cache_dims(kv, kv, 64, 16), None, None)


def test_tokens_of_a_call(L):
    """The kernels step over tokens in 32 bits, a grid's share (2^17) past the last. (An address that is not aligned ends the
    calls that the sizes let through.)"""
    assert tables(L, 2 ** 31 - 1) == tables(L, 2 ** 31 - 2 ** 18) == UNS
    assert tables(L, 2 ** 31 - 2 ** 21) == INV
    assert append(L, 2 ** 31 - 1) == append(L, 2 ** 31 - 200) == UNS
    assert append(L, 2 ** 31 - 2 ** 21) == INV


def test_rows_of_a_cache(L):
    """A page that is none is read past the cache's last row, a box of up to 128 rows in 32 bits."""
    assert append(L, 4, N=(1 << 27) - 1) == UNS and append(L, 4, N=(1 << 27) - 9) == INV


def test_units_of_a_plan_are_summed_within_32_bits():
    """The prompt kernels' plan adds up the units of ranges that the caller's table may let lie over one another, each of up to
    2^31 / 128 rows and 1,024 heads more: its sums, block by block of 32 warps as in csrc/gdn_attn_prefill.cu, stay in
    32 bits and never come out below what the list holds."""
    src = open(os.path.join(build.CSRC, "gdn_attn_prefill.cu")).read()
    assert "carry = min(carry + s_warp[0][i], kManyUnits);" in src and "bv = min(bv + s_warp[0][i], kManyUnits);" in src
    many = 1 << int(re.search(r"kManyUnits = 1 << (\d+);", src).group(1))
    most_of_request = (2 ** 31 - 65536) // 128 + 1024
    largest_list = most_of_request + 1024 * 2048 + 2048 * 3 * 152
    for each in (1, 1000, 2 ** 16, 2 ** 21, most_of_request):
        carry = 0
        for _ in range(2):                        # 2,048 requests, 1,024 at a time
            for _ in range(32):
                assert carry + 32 * each < 2 ** 31
                carry = min(carry + 32 * each, many)
        assert (carry > largest_list) == (2048 * each > largest_list)
