"""What the host tables of rotary positions and their binding refuse."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn
from gated_deltanet_linear_gdn_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def frequencies(rot, base, kind, factor):
    w, f = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    return gdn.lib().gdn_rope_frequencies(rot, base, kind, factor, 0, w, ctypes.byref(f)), list(w)


def test_a_base_that_is_not_finite():
    """NTK-aware scaling multiplies the base by factor^(rot / (rot - 2)): past the largest double there are no frequencies."""
    status, w = frequencies(4, 1e4, gdn.GDN_ROPE_NTK, 1e150)
    assert status == gdn.GDN_OK and w == [1.0, pytest.approx(1e-152, rel=1e-12)]
    assert frequencies(4, 1e4, gdn.GDN_ROPE_NTK, 1e153)[0] == gdn.GDN_ERR_INVALID_ARG
    assert frequencies(64, 1e300, gdn.GDN_ROPE_NTK, 1e10)[0] == gdn.GDN_ERR_INVALID_ARG
    assert frequencies(64, 1e300, gdn.GDN_ROPE_LINEAR, 1e10)[0] == gdn.GDN_OK


def test_an_output_without_its_input():
    q, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_out without k"):
        gdn.gdn_rope(q, None, pos, q, q, gdn.RopeTable(64, device="cpu"))


def test_a_scaling_that_is_none_of_them():
    with pytest.raises(ValueError, match="none, linear, ntk, yarn"):
        gdn.RopeTable(64, scaling="dynamic", device="cpu")
