"""Calls of one kind from several host threads, each with buffers and a stream of its own: what one thread's call asks of a
kernel (its shared memory goes by the batch) does not get into another's."""
import ctypes
import threading

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


def together(calls, times):
    """Each call `times` times on a thread of its own; what they returned. (A call lasts some microseconds without the
    interpreter's lock.)"""
    start, seen = threading.Barrier(len(calls)), [None] * len(calls)

    def loop(i, call):
        start.wait()
        seen[i] = {call() for _ in range(times)}

    threads = [threading.Thread(target=loop, args=(i, c)) for i, c in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def p(t):
    return ctypes.c_void_p(t.data_ptr())


def decode_call(B, keep):
    """A decode call with everything of its own."""
    L, H, Hq, d, bs = gdn.lib(), 1, 2, 64, 16
    cache = torch.zeros(4, H, bs, d, dtype=torch.uint8, device="cuda")
    scale = torch.ones(4, H, device="cuda")
    q = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_attn_decode_workspace_size(B, 1, Hq, H, d, bs), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    keep.extend([cache, scale, q, table, lens, out, ws, stream])
    args = (p(q), Hq * d, p(cache), p(cache), p(scale), p(scale), 4, p(table), 1, p(lens), B, gdn.gdn_cache_dims(Hq, H, d, bs), 0.125,
            p(out), p(ws), ws.numel(), None, ctypes.c_void_p(stream.cuda_stream))
    return lambda: L.gdn_attn_decode(*args)


def test_first_call_of_a_thread():
    """Attention as the first that a host thread asks of CUDA, on a library that is in use already."""
    keep = []
    call = decode_call(3, keep)
    assert call() == gdn.GDN_OK
    torch.cuda.synchronize()
    assert together([call], 3) == [{gdn.GDN_OK}]


def test_decode_batches_of_different_sizes():
    keep = []
    calls = [decode_call(B, keep) for B in (1, 250, 20)]
    torch.cuda.synchronize()
    assert together(calls, 6000) == [{gdn.GDN_OK}] * 3


def test_tables_of_different_sizes():
    L, bs, keep = gdn.lib(), 16, []

    def call(B):
        z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        old, new, table, ring, pool, out, cu, lens = z(B), z(B), z((B, 1)), z(8), z(2), z(2), z(B + 1), z(B)
        stream = torch.cuda.Stream()
        keep.extend([old, new, table, ring, pool, out, cu, lens, stream])
        args = (p(old), p(new), B, p(table), 1, p(ring), 8, p(pool), p(out), bs, 0, p(cu), None, None, p(lens), None,
                ctypes.c_void_p(stream.cuda_stream))
        return lambda: L.gdn_cache_tables(*args)

    torch.cuda.synchronize()
    assert together([call(2600), call(8192), call(4000)], 6000) == [{gdn.GDN_OK}] * 3
