"""mxq_attn with windows up to the largest int32 and sequences with fewer keys than new tokens."""

import pytest
import torch

from test_gpu_attn import Problem, check

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("window,sinks", [(LAST, 0), (LAST, LAST), (LAST - 3, 4), (1, LAST), (600, 0)])
def test_large_windows(mxq, cache, window, sinks):
    """The first tile of a sequence begins before its first key: positions from -20 on, and -1, 0 and above."""
    nq, lens = [60, 3, 4, 1, 2], [40, 3, 3, 500, 0]
    p = Problem(nq, lens, 8, 128, cache, page=16, window=window, sinks=sinks, seed=4000)
    out, lse = p.run(mxq)
    check(out, lse, p.want())
    assert bool((lse[:20] == -float("inf")).all()) and bool(torch.isfinite(lse[20:60]).all())
    assert int(p.err.item()) == 0 and mxq.mxq_watchdog_read() == 0
