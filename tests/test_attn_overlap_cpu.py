"""mxq_attn writes out and lse while other blocks still read the query and the cache: buffers that overlap
are refused, but for out being q itself (a row is read before it is written)."""

import ctypes

import pytest
import torch

T, H, D, SLOTS = 4, 64, 512, 4096
ROWS = T * H * D * 2
Q0, KV0, OUT0, LSE0 = 1 << 30, 1 << 32, 1 << 34, 1 << 36


@pytest.fixture(scope="module")
def L():
    from mxfp8_block_scaled_inv_gb300 import build as B

    B.build()
    import mxfp8_block_scaled_inv_gb300 as mxq

    return mxq.lib()


def attn(L, q=Q0, kv=KV0, out=OUT0, lse=LSE0, dtype=1):
    p = ctypes.c_void_p
    return L.mxq_attn(p(q), T, H, D, None, p(1 << 20), T, p(1 << 21), 8, 64, p(kv), SLOTS, dtype, p(1 << 22),
                      p(1 << 23), 0, 0, 0.1, p(out), p(lse) if lse else None, None, p(1 << 40), 1 << 38, None)


@pytest.mark.parametrize("dtype,row", [(0, D), (1, 2 * D), (2, D // 2)])
def test_overlapping_buffers_are_refused(L, dtype, row):
    lse = T * H * 4
    for bad in (dict(out=Q0 + 16), dict(out=Q0 - 16), dict(out=Q0 + ROWS - 16),
                dict(out=KV0), dict(out=KV0 + SLOTS * row - 16), dict(out=KV0 - ROWS + 16),
                dict(lse=OUT0), dict(lse=OUT0 + ROWS - 4), dict(lse=OUT0 - lse + 4), dict(out=Q0, lse=Q0 + 64),
                dict(lse=Q0), dict(lse=Q0 + ROWS - 4), dict(lse=KV0 + SLOTS * row - 4)):
        assert attn(L, dtype=dtype, **bad) == 2, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("dtype,row", [(0, D), (1, 2 * D), (2, D // 2)])
def test_neighbours_and_in_place_are_accepted(L, dtype, row):
    for good in (dict(), dict(out=Q0), dict(out=Q0 + ROWS), dict(out=Q0 - ROWS), dict(out=KV0 + SLOTS * row),
                 dict(out=KV0 - ROWS), dict(lse=OUT0 + ROWS), dict(lse=Q0 + ROWS), dict(lse=None)):
        assert attn(L, dtype=dtype, **good) == 7, good
