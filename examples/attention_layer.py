"""One attention layer served from a paged KV cache, end to end:

    q, kv -> forward RoPE + insertion into the cache    mxq_rope_kv_insert / mxq_rope_kv4_insert
          -> attention over the pages                   mxq_attn
          -> inverse RoPE, quantisation, wo_a           mxq_wo_a

with the cache in BF16, in E4M3 or in 4 bits.  A chunk of several requests is
prefilled, then every sequence is decoded token by token from a CUDA graph.

    python examples/attention_layer.py
"""

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mxfp8_block_scaled_inv_gb300 as mxq  # noqa: E402


class AttentionLayer:
    """H query heads of D columns over one shared KV row per token (key and value at once), the last R
    columns rotated.  Each head is a group of the projection, N outputs wide."""

    def __init__(self, H=64, D=512, R=64, N=128, cache="e2m1", pages=64, page_size=64, window=0, sinks=0,
                 max_pos=65536, device="cuda", seed=0):
        self.H, self.D, self.R, self.cache_type = H, D, R, cache
        self.page_size, self.window, self.sinks = page_size, window, sinks
        g = torch.Generator().manual_seed(seed)
        angle = torch.arange(max_pos)[:, None] * 10000.0 ** (-torch.arange(0, R, 2)[None] / R)
        self.cos, self.sin = (f(angle).to(torch.bfloat16).to(device) for f in (torch.cos, torch.sin))
        self.w = torch.randn((H, N, D), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(device)
        self.w_sf = mxq.mxq_prepare_weight_scales(
            torch.full((H, N, (D + 127) // 128), 122, dtype=torch.uint8, device=device), D)
        slots = pages * page_size
        self.scale = self.cache_sf = None
        if cache == "bf16":
            self.cache = torch.zeros((slots, D), dtype=torch.bfloat16, device=device)
        elif cache == "e4m3":
            self.cache = torch.zeros((slots, D), dtype=torch.uint8, device=device)
            self.scale = torch.full((1,), 1.0 / 64, device=device)
        else:
            self.cache = torch.zeros((slots, D // 2), dtype=torch.uint8, device=device)
            self.cache_sf = torch.zeros((slots, D // 32), dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def insert(self, q, kv, pos, slots):
        """Rotates q and kv and stores the kv rows; returns the rotated query."""
        if self.cache_type == "e2m1":
            return mxq.mxq_rope_kv4_insert(q, kv, pos, self.cos, self.sin, self.R, slots, self.cache,
                                           self.cache_sf, err_flag=self.err)
        return mxq.mxq_rope_kv_insert(q, kv, pos, self.cos, self.sin, self.R, slots, self.cache, self.scale,
                                      err_flag=self.err)

    def attend(self, q, block_table, seq_lens, q_start=None):
        return mxq.mxq_attn(q, self.cache, block_table, seq_lens, q_start, self.page_size, self.window, self.sinks,
                            kv_scale=self.scale, cache_sf=self.cache_sf, err_flag=self.err)

    def forward(self, q, kv, pos, slots, block_table, seq_lens, q_start=None):
        """q bf16 [T, H, D], kv bf16 [T, D] of T new tokens -> bf16 [T, H, N]."""
        o = self.attend(self.insert(q, kv, pos, slots), block_table, seq_lens, q_start)
        return mxq.mxq_wo_a(o, pos, self.cos, self.sin, self.w, self.w_sf, self.R, err_flag=self.err)


class Requests:
    """Pages, lengths and positions of a batch of sequences: what a scheduler keeps on the host."""

    def __init__(self, layer, batch, max_pages, seed=0):
        self.layer, self.batch = layer, batch
        pages = layer.cache.shape[0] // layer.page_size
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
        self.table = order[:batch * max_pages].reshape(batch, max_pages).to(torch.int32)
        self.lens = [0] * batch

    def append(self, counts):
        """Takes counts[b] more tokens for each sequence; returns positions, cache rows, lengths and starts."""
        ps = self.layer.page_size
        pos, slots, start = [], [], [0]
        for b, n in enumerate(counts):
            for p in range(self.lens[b], self.lens[b] + n):
                pos.append(p)
                slots.append(int(self.table[b, p // ps]) * ps + p % ps)
            self.lens[b] += n
            start.append(len(pos))
        i32 = torch.int32
        return torch.tensor(pos), torch.tensor(slots), torch.tensor(self.lens, dtype=i32), torch.tensor(start, dtype=i32)


def run(cache, chunks=(300, 77, 1), steps=8, seed=0, **layer_args):
    """Prefills one chunk per sequence and decodes `steps` tokens each; returns the layer, its requests, the
    tokens' (q, kv) and the outputs, each a list with the chunk first."""
    layer = AttentionLayer(cache=cache, seed=seed, **layer_args)
    dev, B = layer.cache.device, len(chunks)
    req = Requests(layer, B, layer.cache.shape[0] // layer.page_size // B, seed)
    table = req.table.to(dev)
    g = torch.Generator().manual_seed(seed + 1)

    def tokens(n):
        return (torch.randn((n, layer.H, layer.D), generator=g).to(torch.bfloat16),
                torch.randn((n, layer.D), generator=g).to(torch.bfloat16))

    # The prompts, in one ragged call.
    meta = req.append(chunks)
    given, outs = [tokens(sum(chunks))], []
    q, kv = given[0]
    outs.append(layer.forward(q.to(dev), kv.to(dev), meta[0].to(dev), meta[1].to(dev), table, meta[2].to(dev),
                              meta[3].to(dev)))

    # Decoding: static inputs, captured once, replayed per token.  The first step also runs eagerly, as the
    # warm-up that a capture wants; it writes the same cache rows again.
    static = None
    for _ in range(steps):
        meta = req.append([1] * B)
        given.append(tokens(B))
        step = list(given[-1]) + list(meta[:3])
        if static is None:
            static = [t.to(dev) for t in step]
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                layer.forward(*static[:4], table, static[4])
            torch.cuda.current_stream().wait_stream(stream)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = layer.forward(*static[:4], table, static[4])
        for s, t in zip(static, step):
            s.copy_(t)
        graph.replay()
        outs.append(out.clone())
    torch.cuda.synchronize()
    if int(layer.err) != 0 or mxq.mxq_watchdog_read() != 0:
        raise RuntimeError(f"data errors {int(layer.err)}, watchdog {mxq.mxq_watchdog_read()}")
    return layer, req, given, outs


def main():
    base = None
    for cache in ("bf16", "e4m3", "e2m1"):
        layer, req, _, outs = run(cache, window=128, sinks=4)
        y = torch.cat(outs).float()
        base = y if base is None else base
        bits = {"bf16": 16, "e4m3": 8, "e2m1": 4.25}[cache]
        print(f"{cache:5s} {bits:5} bits a value: {y.shape[0]} tokens, lengths {req.lens}, "
              f"difference from the BF16 cache {float((y - base).norm() / base.norm()):.4f}")


if __name__ == "__main__":
    main()
