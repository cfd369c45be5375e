"""The example that runs the cache calls next to the GDN layer: a request's results do not depend on what is
served with it, and its attention is what plain 64-bit attention over the cache's values gives."""
import os
import sys

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_gdn_gb300 import build
    build.build_library()


def serve(requests, heads, block_size):
    """Each request: (prompt length, decode steps' inputs). Prompts in one step, then a token each, step by step."""
    import hybrid_step as hs
    model = hs.HybridStep(gdn.Dims(2, 4, 128, 128), *heads, block_size=block_size, num_blocks=64,
                          max_requests=4, max_len=1024, max_tokens=1024)
    packed = lambda xs: [torch.cat(x) for x in zip(*xs)]
    lens = torch.tensor([n for n, _, _ in requests], dtype=torch.int32, device="cuda")
    outs = [model.step(*packed([x for _, x, _ in requests]), lens, 0)]
    for t in range(len(requests[0][2])):
        lens = lens + 1
        outs.append(model.step(*packed([x[t] for _, _, x in requests]), lens, len(requests)))
    torch.cuda.synchronize()
    assert int(model.err) == 0
    return model, outs


@pytest.mark.parametrize("heads,block_size", [((8, 2, 128), 16), ((8, 1, 256), 64), ((6, 3, 64), 32)])
def test_hybrid_step(heads, block_size):
    import hybrid_step as hs
    gen = torch.Generator().manual_seed(5)
    shapes = hs.HybridStep(gdn.Dims(2, 4, 128, 128), *heads, max_tokens=64)
    lengths, steps = [131, 1, 64], 3
    requests = [(n, hs.inputs(shapes, n, gen), [hs.inputs(shapes, 1, gen) for _ in range(steps)]) for n in lengths]
    model, together = serve(requests, heads, block_size)
    for i, r in enumerate(requests):
        _, alone = serve([r], heads, block_size)
        first = sum(lengths[:i])
        for got, want in zip([x[first:first + lengths[i]] for x in together[0]], alone[0]):
            assert torch.equal(got, want)
        for t in range(steps):
            for got, want in zip(together[1 + t], alone[1 + t]):
                assert torch.equal(got[i:i + 1], want)

    # the last token of each request against its cache: bf16 rounding of the output (2^-8) and a 16-bit p
    Hq, H, d = heads
    kc, vc, ks, vs = model.cache
    for i, r in enumerate(requests):
        n = lengths[i] + steps
        blocks = model.table[i, :-(-n // block_size)].long()
        k, v = ((c[blocks].double() * s[blocks][:, :, None, None].double()).transpose(1, 2).reshape(-1, H, d)[:n]
                for c, s in ((kc, ks), (vc, vs)))
        q = r[2][-1][3][0, :Hq * d].double().view(H, Hq // H, d)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * d ** -0.5, dim=-1)
        want = torch.einsum("hgn,nhd->hgd", p, v).reshape(Hq, d)
        off = (together[-1][1][i].double() - want).abs()
        assert bool((off <= want.abs() * 2.0 ** -8 + 2.0 ** -12 * v.abs().max()).all())


def test_main(capsys):
    import hybrid_step as hs
    hs.main()
    assert "error word 0" in capsys.readouterr().out
