"""A pool of free blocks that runs short, at sizes from one row on: rows are served in order until a row needs more than is
left; that row and every later one that needs a block keep their length and get no slots. Against the row-by-row restatement."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache_oracle as co

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("old,new,free", [
    ([0], [1], 0), ([5], [40], 1), ([16, 0, 3], [17, 16, 4], 1), ([0, 0, 0], [33, 16, 15], 3), ([40, 16, 20], [0, 30, 21], 0),
    ([10, 32, 0, 7], [80, 33, 0, 8], 4), (list(range(0, 96)), list(range(20, 116)), 60)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_that_are_refused(old, new, free, in_place):
    bs, B = 16, len(old)
    n = -(-np.array(old) // bs)
    used, W, N = int(n.sum()), int((-(-np.maximum(old, new) // bs)).max()) + 1, int(n.sum()) + free + 2
    perm = np.random.default_rng(B).permutation(N)
    table, at = np.full((B, W), -1), 0
    for b in range(B):
        table[b, :n[b]] = perm[at:at + n[b]]
        at += n[b]
    head = N - 1
    ring = np.full(N, -1)
    ring[(head + np.arange(free)) % N] = perm[used:used + free]
    T = int(np.maximum(0, np.subtract(new, old)).sum())
    want = co.tables(old, new, table, ring, [head, free], bs, T)
    assert want["short"]
    d = {"old": i32(old), "new": i32(new), "table": i32(table), "ring": i32(ring), "pool": i32([head, free])}
    z = lambda k: torch.full((k,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {"pool": d["pool"] if in_place else z(2), "cu": z(B + 1), "slots": z(T), "positions": z(T),
           "lens": d["old"] if in_place else z(B), "table": d["table"], "ring": d["ring"]}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_cache_tables(d["old"], d["new"], d["table"], d["ring"], d["pool"], got["pool"], got["cu"], got["slots"], got["positions"],
                         got["lens"], bs, err=err)
    for k in got:
        assert np.array_equal(got[k].cpu().numpy(), want[k]), k
    assert int(err) == gdn.GDN_DEVERR_BLOCKS
