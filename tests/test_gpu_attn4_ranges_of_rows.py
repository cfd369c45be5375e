"""Prompts over the 4-bit cache whose cu_tokens are not a step's: a request outside the rows counts as empty, for the room of the
others' pages too."""
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

from test_gpu_attn4 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("first", [-5, -0x80000000])
def test_a_request_that_starts_before_the_first_row(first):
    c = Case(3, [20, 30, 7], [100, 50, 60], 4, 2, 64, 16)            # 8, 5 and 5 blocks
    good, rows = c.prefill(), c.cu.tolist()
    c.cu[0] = first
    got = c.prefill(held=10)
    assert int(c.err) == gdn.GDN_DEVERR_SEQLENS
    assert torch.equal(got[rows[1]:], good[rows[1]:]) and bool((got[:rows[1]] == 5.0).all())


@pytest.mark.parametrize("end", [58, 0x7fffffff])
def test_requests_that_end_behind_the_last_row(end):
    c = Case(4, [20, 30, 7], [100, 50, 60], 4, 2, 64, 16)
    good, rows = c.prefill(), c.cu.tolist()
    c.cu[3] = end                                                   # (57 rows)
    got = c.prefill(held=13)
    assert int(c.err) == gdn.GDN_DEVERR_SEQLENS
    assert torch.equal(got[:rows[2]], good[:rows[2]]) and bool((got[rows[2]:] == 5.0).all())


def test_a_request_in_the_middle():
    """(cu_tokens that go down: the range before is too long, the one after starts late.)"""
    c = Case(5, [20, 30, 7], [100, 50, 60], 4, 2, 64, 16)
    good, rows = c.prefill(), c.cu.tolist()
    c.cu[2] = 1000
    got = c.prefill(held=8)
    assert int(c.err) == gdn.GDN_DEVERR_SEQLENS
    assert torch.equal(got[:rows[1]], good[:rows[1]]) and bool((got[rows[1]:] == 5.0).all())
