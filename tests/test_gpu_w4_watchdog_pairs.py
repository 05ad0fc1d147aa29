"""Waits of the pair form of the 4-bit products that run out: the kernel waits for every copy that it issued, and for no
more than these.  (A barrier that lacks an arrival or bytes would hold it for the two seconds that such a wait may
take; one that got too many would let go early and spoil the next phase.)"""

import time

import pytest
import torch

from test_gpu_w4_watchdog import BIT, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def expire(mxq, call, times):
    want = call().clone()
    torch.cuda.synchronize()
    assert mxq.mxq_watchdog_read(clear=True) == 0
    for ns in times:
        mxq.mxq_debug_set_w4_wait(ns)
        try:
            began = time.perf_counter()
            call()
            torch.cuda.synchronize()
            took = time.perf_counter() - began
        finally:
            mxq.mxq_debug_set_w4_wait(0)
        assert mxq.mxq_watchdog_read(clear=True) in (0, BIT)
        assert took < 1.0, took
        assert torch.equal(call(), want)
        torch.cuda.synchronize()
        assert mxq.mxq_watchdog_read() == 0


TIMES = [1000, 1000, 2000, 3000, 5000, 8000, 13000, 21000, 50000]


@pytest.mark.parametrize("T,N,K", [(600, 32768, 65536), (240, 16384, 65536), (417, 32768, 16384), (1000, 20464, 8192)])
def test_linear(mxq, T, N, K):
    w4 = mxq.mxq_prepare_w4(*tensors((N,), K, 1, 32))
    a, sf = tensors((T,), K, 2, 128)
    expire(mxq, lambda: mxq.mxq_linear_a8w4(a, sf, w4, N), TIMES)


@pytest.mark.parametrize("T,k,E", [(900, 4, 16), (700, 4, 13)])
def test_experts(mxq, T, k, E):
    """Tiles of different sizes one behind the other, whose stages have different numbers of bytes."""
    K, I = 16384, 1024
    w13 = mxq.mxq_prepare_w4(*tensors((2 * E, I), K, 3, 32))
    w2 = mxq.mxq_prepare_w4(*tensors((E, K), I, 4, 32))
    a, sf = tensors((T,), K, 5, 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    ids = (torch.rand((T, k), generator=g, device="cuda") ** 2 * E).int().clamp_(0, E - 1)
    wt = torch.full((T, k), 0.25, device="cuda")
    expire(mxq, lambda: mxq.mxq_experts_a8w4(a, sf, ids, wt, w13, w2, I), TIMES)
