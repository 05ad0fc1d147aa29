"""mxq_attn with as many new tokens as sequences, but not one each: q_start decides,
with the workspace that the size query names."""

import numpy as np
import pytest
import torch

from test_gpu_attn import Problem, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("B,H,D,top", [(131, 1, 64, 4000), (160, 20, 128, 700), (31, 40, 128, 1500), (9, 64, 256, 900)])
@pytest.mark.parametrize("ragged", [False, True])
def test_as_many_tokens_as_sequences(mxq, cache, B, H, D, top, ragged):
    rng = np.random.Generator(np.random.PCG64(B))
    lens = [int(v) for v in rng.integers(1, top, B)]
    lens[0] = top
    nq = [1] * B
    if ragged:
        nq[1::3] = [3 if 3 * i + 2 < B else 1 for i in range(len(nq[1::3]))]
        for b in range(1, B - 1, 3):
            nq[b - 1] = nq[b + 1] = 0
        nq[-1] += B - sum(nq)
    assert sum(nq) == B
    lens = [max(n, l) for n, l in zip(nq, lens)]
    p = Problem(nq, lens, H, D, cache, page=64, seed=2000 + B)
    out, lse = p.run(mxq)
    check(out, lse, p.want())
    assert int(p.err.item()) == 0 and mxq.mxq_watchdog_read() == 0
    if not ragged:
        # The same without q_start, the workspace given.
        d = "cuda"
        need = mxq.mxq_attn_workspace_bytes(B, B, H, D, p.pages, 64)
        out = mxq.mxq_attn(p.q.to(d), p.kv.to(d), torch.from_numpy(p.bt).to(d),
                           torch.tensor(lens, dtype=torch.int32, device=d), kv_scale=torch.tensor([0.0371], device=d),
                           cache_sf=None if p.sf is None else p.sf.to(d),
                           ws=torch.empty(need, dtype=torch.uint8, device=d) if need else None)
        check(out, None, p.want())
