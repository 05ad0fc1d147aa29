"""The example that runs the cache operators together: insertion, attention and
projection, prefilled in one ragged chunk and decoded from a CUDA graph."""

import os
import sys

import numpy as np
import pytest

import attn_ref as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import attention_layer
    finally:
        sys.path.pop(0)
    return attention_layer


def cache_rows(layer):
    """What the cache holds, in 64 bits."""
    c = layer.cache.cpu()
    if layer.cache_type == "bf16":
        return c.double().numpy()
    if layer.cache_type == "e4m3":
        return A.e4m3_values(c.numpy()) * float(layer.scale)
    return A.e2m1_values(c.numpy(), layer.cache_sf.cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_layer(example, cache, window, sinks):
    """Chunk and decode steps agree with a fresh pass over the finished cache, that pass's attention with the
    64-bit reference, and the cache with what was inserted."""
    import torch

    import mxfp8_block_scaled_inv_gb300 as mxq

    chunks, steps = (70, 9, 1), 3
    layer, req, given, outs = example.run(cache, chunks, steps, seed=5, H=16, D=128, R=64, N=64, pages=15,
                                          page_size=16, window=window, sinks=sinks, max_pos=256)
    B, dev = len(chunks), layer.cache.device
    rows = cache_rows(layer)

    # The new tokens again, in one call: the same rows are written, and the same keys are seen.
    want = []
    again = example.Requests(layer, B, req.table.shape[1], 5)
    counts = [c + steps for c in chunks]
    pos, slots, lens, start = again.append(counts)
    q = torch.empty((len(pos), layer.H, layer.D), dtype=torch.bfloat16)
    kv = torch.empty((len(pos), layer.D), dtype=torch.bfloat16)
    first = np.concatenate([[0], np.cumsum(chunks)])
    for b in range(B):
        s, n = int(start[b]), chunks[b]
        q[s:s + n], kv[s:s + n] = given[0][0][first[b]:first[b] + n], given[0][1][first[b]:first[b] + n]
        want.append(outs[0][first[b]:first[b] + n])
        for i in range(steps):
            q[s + n + i], kv[s + n + i] = given[1 + i][0][b], given[1 + i][1][b]
            want.append(outs[1 + i][b:b + 1])
    want = torch.cat(want).double().cpu().numpy()
    q_rot = layer.insert(q.to(dev), kv.to(dev), pos.to(dev), slots.to(dev))
    assert np.array_equal(cache_rows(layer), rows)
    table = req.table.to(dev)
    o = layer.attend(q_rot, table, lens.to(dev), start.to(dev))
    ref, _, mag, sabs = A.attention(q_rot.double().cpu().numpy(), rows, req.table.numpy(), layer.page_size,
                                    start.numpy(), lens.numpy(), window, sinks, layer.D ** -0.5)
    # Weights and output rounded to BF16 or better, 2^-9 each, and scores within 2^-19 of their products' sizes;
    # twice that is allowed.
    tol = mag * (2.0 ** -7 + 2.0 ** -17 * sabs[..., None]) + 1e-30
    assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()

    # The projection quantises o to E4M3: a step of its codes is 2^-3 of a value at most, and o differs by an
    # ulp of BF16 between the two runs where sums are split differently.  Both have the same expected value, so
    # the norms of the rows are compared: 128 values with independent steps of 2^-4 on average.
    y = mxq.mxq_wo_a(o, pos.to(dev), layer.cos, layer.sin, layer.w, layer.w_sf, layer.R).double().cpu().numpy()
    err = np.linalg.norm(y - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), 1e-30)
    assert err.max() <= 2.0 ** -4
