"""The calls whose arguments are marshalled in C++, from several host threads at once, each with its own stream, buffers and
workspace; the first of them meet a binding that is not loaded yet."""
import threading

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

from test_gpu_attn4 import Case

pytestmark = pytest.mark.gpu

THREADS, TURNS = 6, 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()
    assert torch.cuda.is_available()


class Step:
    """One thread's buffers: positions, write, read-back and both attentions, of sizes that differ from the other threads'."""

    def __init__(self, i):
        d, bs, H, G = (64, 128, 256)[i % 3], (16, 64)[i % 2], 1 + i % 3, (1, 4, 8)[i // 2 % 3]
        self.one = Case(i, [1] * (3 + i), [50 * (j + 1) for j in range(3 + i)], H * G, H, d, bs)
        self.many = Case(50 + i, [20 + i, 7], [100, 0], H * G, H, d, bs)
        self.rope = gdn.RopeTable(d // 2, base=1e5)
        T = self.many.T
        g = torch.Generator().manual_seed(i)
        self.k = torch.randn(T, H, d, generator=g).bfloat16().cuda()
        self.pos = torch.randint(0, 10000, (T,), generator=g).int().cuda()
        blocks = self.many.cache[0].shape[0]
        self.slots = torch.randperm(blocks * bs, generator=g)[:T].int().cuda()
        self.fresh = [x.clone() for x in self.many.cache]

    def run(self):
        kk, out = torch.empty_like(self.k), torch.empty(2, *self.k.shape, dtype=torch.bfloat16, device="cuda")
        cache = [x.clone() for x in self.fresh]
        gdn.gdn_rope(self.many.q, self.k, self.pos, torch.empty_like(self.many.q), kk, self.rope)
        gdn.gdn_cache4_append(kk, self.k, self.slots, *cache)
        gdn.gdn_cache4_read(*cache, self.slots, out[0], out[1])
        return [kk, out, *cache, self.one.decode(), self.many.prefill()]


def test_threads(monkeypatch):
    steps = [Step(i) for i in range(THREADS)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    monkeypatch.setattr(gdn, "_marshal", None)
    start, wrong = threading.Barrier(THREADS), []

    def serve(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(TURNS):
                    got = steps[i].run()
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 (the test's own thread shows it)
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=serve, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for s in steps:
        assert int(s.one.err) == 0 and int(s.many.err) == 0


def test_refusals_of_one_thread_leave_the_others(monkeypatch):
    """A thread whose calls raise, next to one whose calls run."""
    s, t, wrong = Step(1), Step(4), []
    want = s.run()
    torch.cuda.synchronize()
    done = threading.Event()

    def refused():
        while not done.is_set():
            try:
                gdn.gdn_cache4_append(t.k, t.k[:-1], t.slots, *t.fresh)
                wrong.append("not refused")
            except ValueError as e:
                if "v must be" not in str(e):
                    wrong.append(str(e))

    other = threading.Thread(target=refused)
    other.start()
    try:
        for _ in range(TURNS):
            got = s.run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        done.set()
        other.join()
    assert not wrong
