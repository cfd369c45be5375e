"""The example's step with positions and the 4-bit cache: a request's results do not depend on what is served with it,
its attention is what plain 64-bit attention over the cache's values gives, and the cache holds its turned keys."""
import os
import sys

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

import _cache4_oracle as co

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()


def serve(requests, heads, block_size, rope):
    """Each request: (prompt length, its inputs, decode steps' inputs). Prompts in one step, then a token each."""
    import hybrid_step as hs
    model = hs.HybridStep(gdn.Dims(2, 4, 128, 128), *heads, block_size=block_size, num_blocks=64, max_requests=4, max_len=1024,
                          max_tokens=1024, cache_bits=4, rope=rope)
    packed = lambda xs: [torch.cat(x) for x in zip(*xs)]  # noqa: E731
    lens = torch.tensor([n for n, _, _ in requests], dtype=torch.int32, device="cuda")
    outs = [model.step(*packed([x for _, x, _ in requests]), lens, 0)]
    for t in range(len(requests[0][2])):
        lens = lens + 1
        outs.append(model.step(*packed([x[t] for _, _, x in requests]), lens, len(requests)))
    torch.cuda.synchronize()
    assert int(model.err) == 0
    return model, outs


@pytest.mark.parametrize("heads,block_size,rot", [((8, 2, 128), 16, 128), ((8, 1, 256), 64, 64), ((6, 3, 64), 32, 20)])
def test_step(heads, block_size, rot):
    import hybrid_step as hs
    gen = torch.Generator().manual_seed(6)
    rope = gdn.RopeTable(rot, base=1e6)
    shapes = hs.HybridStep(gdn.Dims(2, 4, 128, 128), *heads, max_tokens=64)
    lengths, steps = [131, 1, 64], 3
    requests = [(n, hs.inputs(shapes, n, gen), [hs.inputs(shapes, 1, gen) for _ in range(steps)]) for n in lengths]
    model, together = serve(requests, heads, block_size, rope)
    for i, r in enumerate(requests):
        _, alone = serve([r], heads, block_size, rope)
        first = sum(lengths[:i])
        for got, want in zip([x[first:first + lengths[i]] for x in together[0]], alone[0]):
            assert torch.equal(got, want)
        for t in range(steps):
            for got, want in zip(together[1 + t], alone[1 + t]):
                assert torch.equal(got[i:i + 1], want)

    Hq, H, d = heads
    k, v = co.unpack(*model.cache)
    last = torch.cat([r[2][-1][3] for r in requests])
    n = torch.tensor([x + steps for x in lengths], dtype=torch.int32, device="cuda")
    q = torch.empty(3, Hq, d, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_rope(last[:, :Hq * d].unflatten(1, (Hq, d)), None, n - 1, q, None, rope)
    want, tol = co.attention(q, None, k, v, model.table[:3], n, d ** -0.5, 11, 2.0 ** -34)
    assert bool(((together[-1][1].double() - want).abs() <= tol).all())
    # the first tokens' keys, turned by their positions, to half a step of their groups
    for i, (length, x, _) in enumerate(requests):
        raw = x[3][:, Hq * d:(Hq + H) * d].unflatten(1, (H, d))
        pos = torch.arange(length, device="cuda")
        turned, _ = co.rope(raw, pos, rope.freqs, 1.0, rot, False)
        held = k[model.table[i, pos // block_size].long(), :, pos % block_size].unflatten(-1, (-1, 32))
        turned = turned.unflatten(-1, (-1, 32))
        # half the step of 2 at 4 to 6, of a scale that the largest is more than 3.5 times of; and the rounding to bf16
        assert bool(((held - turned).abs() <= turned.abs().amax(dim=-1, keepdim=True) * (2 / 7 + 2.0 ** -7)).all())
