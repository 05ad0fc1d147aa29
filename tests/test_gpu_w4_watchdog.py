"""Waits of the 4-bit products that run out, without faulting the GPU: every wait is bounded to a microsecond
(32 tries, some hundred in effect), and a gigabyte of weights keeps the epilogue's first wait longer.  The kernels
set their watchdog bit, let what they issued end and return; later calls give the same bits as ever."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BIT = 0x80


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def tensors(shape, K, seed, group):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = 2 if group == 32 else 1
    c = torch.randint(0, 0x70, (*shape, K // per), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(115, 122, (*shape, -(-K // group)), generator=g, device="cuda", dtype=torch.uint8)
    return c, s


def expire(mxq, call):
    want = call().clone()
    torch.cuda.synchronize()
    assert mxq.mxq_watchdog_read(clear=True) == 0
    for _ in range(3):
        assert mxq.mxq_debug_set_w4_wait(1000) == 2_000_000_000
        try:
            call()  # returns: the kernels gave up instead of hanging
            torch.cuda.synchronize()
        finally:
            assert mxq.mxq_debug_set_w4_wait(0) == 1000
        assert mxq.mxq_watchdog_read(clear=True) == BIT
        assert torch.equal(call(), want)
        torch.cuda.synchronize()
        assert mxq.mxq_watchdog_read() == 0


@pytest.mark.parametrize("T", [1, 32, 48, 100, 600])
def test_linear(mxq, T):
    """Split K over clusters, streaming CTAs, CTA pairs."""
    N, K = 32768, 65536
    w4 = mxq.mxq_prepare_w4(*tensors((N,), K, 1, 32))
    a, sf = tensors((T,), K, 2, 128)
    expire(mxq, lambda: mxq.mxq_linear_a8w4(a, sf, w4, N))


@pytest.mark.parametrize("T,k,E", [(4, 4, 16), (8, 4, 16), (100, 4, 16), (200, 4, 16), (900, 4, 16)])
def test_experts(mxq, T, k, E):
    K, I = 65536, 1024
    w13 = mxq.mxq_prepare_w4(*tensors((2 * E, I), K, 3, 32))
    w2 = mxq.mxq_prepare_w4(*tensors((E, K), I, 4, 32))
    a, sf = tensors((T,), K, 5, 128)
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) % E
    wt = torch.full((T, k), 0.25, device="cuda")
    expire(mxq, lambda: mxq.mxq_experts_a8w4(a, sf, ids, wt, w13, w2, I))
