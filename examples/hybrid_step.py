"""A serving step of a hybrid model: a GDN layer with its recurrent states next to an attention layer with its
8-bit paged cache, for a batch of decode rows followed by prompts.

    python examples/hybrid_step.py          # prompts, then decode steps replayed as one CUDA graph

The library works between a layer's projections, so a step takes what those give (random here): the GDN layer's
packed q | k | v channels and gates, the attention layer's q, k and v.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_gdn_gb300 as gdn  # noqa: E402

I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32


class HybridStep:
    """States, cache and workspaces of up to max_requests requests; row r of a step is request r."""

    def __init__(self, dims, q_heads, kv_heads, head_dim, *, block_size=64, num_blocks=256, max_requests=8,
                 max_len=4096, max_tokens=4096, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        new = lambda *shape, dtype=F32: torch.zeros(*shape, dtype=dtype, device=device)
        self.dims, self.heads = dims, (q_heads, kv_heads, head_dim)
        # GDN layer: weights, one recurrent and one conv state per slot (slot 0 is the null slot)
        self.A_log = torch.rand(dims.Hv, generator=g).to(device)
        self.dt_bias = torch.rand(dims.Hv, generator=g).to(device)
        self.conv_weight = (torch.randn(dims.D, dims.W, generator=g) / dims.W).to(BF16).to(device)
        self.conv_state = new(max_requests + 1, dims.D, dims.W - 1, dtype=BF16)
        self.ssm = new(max_requests + 1, dims.Hv, dims.dv, dims.dk)
        self.slot = torch.arange(1, max_requests + 1, dtype=I32, device=device)
        # attention layer: the cache, its free blocks, a table row per request
        self.block_size = block_size
        self.cache = (new(num_blocks, kv_heads, block_size, head_dim, dtype=torch.float8_e4m3fn),
                      new(num_blocks, kv_heads, block_size, head_dim, dtype=torch.float8_e4m3fn),
                      new(num_blocks, kv_heads), new(num_blocks, kv_heads))
        self.free = torch.arange(num_blocks, dtype=I32, device=device)
        self.pool = torch.tensor([0, num_blocks], dtype=I32, device=device)
        width = -(-max_len // block_size)
        self.table = new(max_requests, width, dtype=I32)
        self.lens = new(max_requests, dtype=I32)
        self.err = new(1, dtype=I32)
        byte = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device=device)
        self.ws_gdn = byte(gdn.gdn_chunked_prefill_workspace_size(max_tokens, max_requests, dims))
        self.ws_attn = byte(max(
            gdn.gdn_attn_decode_workspace_size(max_requests, width, *self.heads, block_size),
            gdn.gdn_attn_prefill_workspace_size(max_tokens, max_requests, width, *self.heads, block_size)))

    def step(self, mixed, a, b, qkv, lens_new, num_decode):
        """mixed [T, D], a and b [T, Hv]: the GDN layer's; qkv [T, (Hq + 2 Hkv) d]: the attention layer's. Row r is to
        hold lens_new[r] tokens; rows before num_decode gain one, the others are prompts. Both layers' outputs."""
        (T, _), (rows,), nd = mixed.shape, lens_new.shape, num_decode
        Hq, H, d = self.heads
        cu = torch.empty(rows + 1, dtype=I32, device=mixed.device)
        slots, positions = torch.empty(2, T, dtype=I32, device=mixed.device)
        lens, table = self.lens[:rows], self.table[:rows]
        gdn.gdn_cache_tables(lens, lens_new, table, self.free, self.pool, self.pool, cu, slots, positions, lens,
                             self.block_size, err=self.err)

        core = torch.empty(T, self.dims.Hv, self.dims.dv, dtype=BF16, device=mixed.device)
        fresh = torch.zeros(rows - nd, dtype=torch.uint8, device=mixed.device)  # prompts begin from nothing
        gdn.gdn_mixed_step(mixed, a, b, self.A_log, self.dt_bias, self.conv_weight, None, self.conv_state, self.ssm,
                           self.slot[:rows], nd, cu[nd:] - nd, fresh, core, self.ws_gdn, self.dims, err=self.err)

        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, H * d, H * d], dim=1))
        out = torch.empty(T, Hq, d, dtype=BF16, device=mixed.device)
        gdn.gdn_cache_append(k, v, slots, *self.cache, err=self.err)
        if nd:
            gdn.gdn_attn_decode(q[:nd], *self.cache, table[:nd], lens[:nd], out[:nd], self.ws_attn, err=self.err)
        if rows > nd:
            gdn.gdn_attn_prefill(q, cu[nd:], *self.cache, table[nd:], lens[nd:], out, self.ws_attn, err=self.err)
        return core, out


def inputs(model, tokens, generator, device="cuda"):
    """What the two layers' input projections would give for `tokens` tokens."""
    Hq, H, d = model.heads
    sizes = (model.dims.D, model.dims.Hv, model.dims.Hv, (Hq + 2 * H) * d)
    return [torch.randn(tokens, n, generator=generator).to(BF16).to(device) for n in sizes]


def main():
    gen = torch.Generator().manual_seed(1)
    model = HybridStep(gdn.Dims(16, 32, 128, 128), 16, 2, 256)
    prompts = [700, 33, 1500, 256]
    lens = torch.tensor(prompts, dtype=I32, device="cuda")
    core, out = model.step(*inputs(model, sum(prompts), gen), lens, 0)
    print("prompts:", tuple(core.shape), tuple(out.shape))

    buffers = inputs(model, len(prompts), gen)
    decode = lambda: model.step(*buffers, model.lens[:len(prompts)] + 1, len(prompts))
    decode()  # (the first call of each kind sets its kernels up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        core, out = decode()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 100
    start.record()
    for _ in range(steps):
        for x in buffers:   # the next token's projections go where the graph reads
            x.copy_(torch.roll(x, 1, 1))
        graph.replay()
    stop.record()
    stop.synchronize()
    print(f"decode: {start.elapsed_time(stop) / steps * 1e3:.1f} us a step of {len(prompts)} rows, lengths",
          model.lens[:len(prompts)].tolist(), "error word", int(model.err))


if __name__ == "__main__":
    main()
