"""mxq_attn with out being the query itself: the same bits as out of place, whole tiles and keys split over CTAs."""

import pytest
import torch

from test_gpu_attn import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("nq,lens,H,D,window", [([1, 1], [3000, 40], 16, 512, 0), ([300, 1, 30], [400, 90, 30], 5, 64, 0),
                                                ([2500], [2500], 33, 128, 50)])
def test_in_place(mxq, cache, nq, lens, H, D, window):
    p = Problem(nq, lens, H, D, cache, window=window, sinks=2, seed=6000 + H)
    want, lse = p.run(mxq)
    # Off by 16 bytes, so that neighbouring rows share sectors.
    buf = torch.zeros(p.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    q = buf[8:].view(p.q.shape)
    q.copy_(p.q)
    host, p.q = p.q, type("Q", (), {"to": lambda s, d: q, "shape": p.q.shape})()
    out, lse2 = p.run(mxq, out=q)
    p.q = host
    assert out.data_ptr() == q.data_ptr()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, lse2)
    assert mxq.mxq_watchdog_read() == 0
