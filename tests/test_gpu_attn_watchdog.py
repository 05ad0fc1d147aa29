"""Waits of the attention kernel that run out, without faulting the GPU: every wait is bounded to a
microsecond (two tries, 8 us, in effect) in batches where the warp that hands out the work has to walk past
tens of thousands of sequences without tokens between two items.  The others give up on the next item, some
before their first, some with copies and products of the last one under way.  The kernel sets its watchdog
bit and returns; later calls give the same bits as ever."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BIT = 0x40


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("tokens,length,H", [(1, 3000, 64), (3, 900, 5), (4, 700, 8), (640, 1000, 64)])
def test_waits_that_run_out(mxq, cache, tokens, length, H):
    """The first and the last of 60000 sequences have tokens; few of them (keys in equal shares over the
    CTAs) or 1280 tiles (whole tiles)."""
    B, D, page, d = 60000, 512, 64, "cuda"
    pages = -(-length // page)
    g = torch.Generator(device=d)
    g.manual_seed(5000)
    q = torch.randn((2 * tokens, H, D), generator=g, device=d).bfloat16()
    x = torch.randn((pages * page, D), generator=g, device=d)
    kw = {}
    if cache == "bf16":
        kv = x.bfloat16()
    elif cache == "e4m3":
        kv = (x * 20.0).to(torch.float8_e4m3fn).view(torch.uint8)
        kw["kv_scale"] = torch.tensor([0.05], device=d)
    else:
        kv = torch.randint(0, 256, (pages * page, D // 2), generator=g, device=d, dtype=torch.uint8)
        kw["cache_sf"] = torch.full((pages * page, D // 32), 126, dtype=torch.uint8, device=d)
    bt = torch.arange(pages, dtype=torch.int32, device=d).expand(B, -1).contiguous()
    lens = torch.full((B,), length, dtype=torch.int32, device=d)
    start = np.full(B + 1, tokens, np.int32)
    start[0], start[B] = 0, 2 * tokens
    kw.update(q_start=torch.from_numpy(start).to(d), page_size=page)

    def call():
        lse = torch.empty(q.shape[:2], device=d)
        out = mxq.mxq_attn(q, kv, bt, lens, lse=lse, **kw)
        torch.cuda.synchronize()
        return out.view(torch.int16), lse

    out, lse = call()
    assert mxq.mxq_watchdog_read(clear=True) == 0 and bool(torch.isfinite(lse).all())
    for _ in range(3):
        assert mxq.mxq_debug_set_attn_wait(1000) == 2_000_000_000
        try:
            call()  # returns: the kernel gave up instead of hanging
        finally:
            assert mxq.mxq_debug_set_attn_wait(0) == 1000
        assert mxq.mxq_watchdog_read(clear=True) == BIT
        again, lse2 = call()
        assert torch.equal(again, out) and torch.equal(lse2, lse)
        assert mxq.mxq_watchdog_read() == 0
