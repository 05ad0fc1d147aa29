"""mxq_prepare_w4 byte for byte, and mxq_linear_a8w4 against 64-bit products: |y - y_ref| <= 1 bf16 ulp(y_ref)
+ 1e-5 * sum_k |a_k w_k|, the rule of the library's other products."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
from cases import check_gemm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def weight(shape, K, seed, lo=118, hi=124):
    g = rng(seed)
    return (g.integers(0, 256, (*shape, K // 2), dtype=np.uint8),
            g.integers(lo, hi, (*shape, K // 32), dtype=np.uint8))


def acts(T, K, seed, lo=115, hi=122):
    g = rng(seed)
    a = g.integers(0, 256, (T, K), dtype=np.uint8)
    a[(a & 0x7F) == 0x7F] = 0x38  # no NaN codes
    return a, g.integers(lo, hi, (T, -(-K // 128)), dtype=np.uint8)


def dev(*x):
    return [torch.from_numpy(v).cuda() for v in x]


def blocks(w, sf):
    """[B, N, K/2], [B, N, K/32] -> the documented layout, element by element."""
    B, N, half = w.shape
    NB, KB = -(-N // 128), -(-half // 64)
    pw = np.zeros((B, NB * 128, KB * 64), np.uint8)
    ps = np.full((B, NB * 128, KB * 4), 127, np.uint8)
    pw[:, :N, :half], ps[:, :N, :half // 16] = w, sf
    out = np.zeros((B, NB, KB, 8704), np.uint8)
    for nb in range(NB):
        for kb in range(KB):
            c = pw[:, nb * 128:nb * 128 + 128, kb * 64:kb * 64 + 64]
            out[:, nb, kb, :8192] = c.reshape(B, 8192)
            for r in range(128):
                at = 8192 + 16 * (r % 32) + 4 * (r // 32)
                out[:, nb, kb, at:at + 4] = ps[:, nb * 128 + r, kb * 4:kb * 4 + 4]
    return out.reshape(-1)


@pytest.mark.parametrize("B,N,K", [(1, 1, 32), (1, 128, 128), (2, 130, 288), (3, 200, 576), (1, 1024, 4096)])
def test_layout(mxq, B, N, K):
    w, sf = weight((B, N), K, seed=B * N + K)
    got = mxq.mxq_prepare_w4(*dev(w, sf)).cpu().numpy()
    assert np.array_equal(got, blocks(w, sf))


def run(mxq, T, N, K, seed, **kw):
    w, wsf = weight((N,), K, seed)
    a, asf = acts(T, K, seed + 1, **kw)
    w4 = mxq.mxq_prepare_w4(*dev(w, wsf))
    out = mxq.mxq_linear_a8w4(*dev(a, asf), w4, N)
    torch.cuda.synchronize()
    assert mxq.mxq_watchdog_read() == 0
    y, S = ref.linear(ref.act_values(a, asf), ref.weight_values(w, wsf))
    check_gemm(out, y, S, f"T={T} N={N} K={K}")
    return out


@pytest.mark.parametrize("N,K", [(16, 32), (128, 128), (144, 160), (1024, 288), (5120, 576), (1024, 4096), (2304, 1152),
                                 (256, 8192)])
@pytest.mark.parametrize("T", [1, 2, 7, 15, 16, 17, 32, 33, 48, 64])
def test_few_tokens(mxq, T, N, K):
    run(mxq, T, N, K, seed=T + N + K)


@pytest.mark.parametrize("T,N,K", [(65, 272, 96), (100, 1024, 576), (127, 4096, 256), (128, 128, 4096), (129, 144, 1024),
                                   (255, 1040, 352), (256, 2048, 1024), (257, 512, 640), (1000, 368, 288),
                                   (2049, 256, 160), (513, 1024, 2048)])
def test_many_tokens(mxq, T, N, K):
    run(mxq, T, N, K, seed=T + N + K)


def test_rows_do_not_depend_on_the_batch(mxq):
    """A token alone, and the same token among others of its launch shape, give the same bits."""
    N, K = 1024, 1152
    w4 = mxq.mxq_prepare_w4(*dev(*weight((N,), K, seed=40)))
    a, asf = dev(*acts(16, K, seed=41))
    all_ = mxq.mxq_linear_a8w4(a, asf, w4, N)
    for t in (0, 5, 15):
        one = mxq.mxq_linear_a8w4(a[t:t + 1].clone(), asf[t:t + 1].clone(), w4, N)
        assert torch.equal(one[0], all_[t])


def test_every_code_and_extreme_scales(mxq):
    """All pairs of codes; scales whose products span 2^-100 to 2^100."""
    K, N, T = 256, 32, 16
    w = np.zeros((N, K // 2), np.uint8)
    for n in range(N):
        w[n] = (n % 16) | ((n * 7 % 16) << 4)
    a = np.tile(np.arange(256, dtype=np.uint8), (T, 1))
    a[(a & 0x7F) == 0x7F] = 0
    wsf = np.full((N, K // 32), 127, np.uint8)
    asf = np.full((T, 2), 127, np.uint8)
    wsf[16:24], wsf[24:] = 77, 177
    asf[4:8], asf[8:12] = 77, 177
    asf[12:, 1] = 100
    wsf[::2, 3] = 120
    out = mxq.mxq_linear_a8w4(*dev(a, asf), mxq.mxq_prepare_w4(*dev(w, wsf)), N)
    y, S = ref.linear(ref.act_values(a, asf), ref.weight_values(w, wsf))
    check_gemm(out, y, S, "codes")


def test_nan_stays_in_its_row_and_column(mxq):
    for T in (16, 40, 130):
        N, K = 144, 288
        w, wsf = weight((N,), K, seed=50)
        a, asf = acts(T, K, seed=51)
        good = mxq.mxq_linear_a8w4(*dev(a, asf), mxq.mxq_prepare_w4(*dev(w, wsf)), N)
        a[3, 17] = 0x7F           # a NaN code
        asf[11, 2] = 0xFF         # a NaN scale
        wsf[100, 5] = 0xFF
        out = mxq.mxq_linear_a8w4(*dev(a, asf), mxq.mxq_prepare_w4(*dev(w, wsf)), N)
        nan = torch.isnan(out)
        want = torch.zeros_like(nan)
        want[3], want[11], want[:, 100] = True, True, True
        assert torch.equal(nan, want)
        assert torch.equal(out[~want], good[~want])


def test_sliced_rows_and_given_output(mxq):
    """Scale rows at an odd address, an output inside a larger buffer whose neighbours stay."""
    N, K, T = 256, 1152, 21
    w4 = mxq.mxq_prepare_w4(*dev(*weight((N,), K, seed=60)))
    a, asf = dev(*acts(T + 2, K, seed=61))
    want = mxq.mxq_linear_a8w4(a[1:T + 1].clone(), asf[1:T + 1].clone(), w4, N)
    buf = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.mxq_linear_a8w4(a[1:T + 1], asf[1:T + 1], w4, N, out=buf[1:T + 1])
    assert torch.equal(buf[1:T + 1], want)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


def test_streams_and_graph(mxq):
    """On a side stream, and captured and replayed on new activations, behind the quantiser that makes them."""
    N, K = 1024, 576
    w4 = mxq.mxq_prepare_w4(*dev(*weight((N,), K, seed=70)))
    g = torch.Generator(device="cuda")
    for T in (1, 20, 50, 200):
        g.manual_seed(T)
        x = torch.randn((3, T, 1, K), generator=g, device="cuda").bfloat16()
        want = []
        for i in range(3):
            q, sc = mxq.mxq_inv_rope_group_quant(x[i])
            want.append(mxq.mxq_linear_a8w4(q.view(T, K), sc.view(T, -1), w4, N))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        q, sc = mxq.mxq_inv_rope_group_quant(x[0], stream=side)
        got = mxq.mxq_linear_a8w4(q.view(T, K), sc.view(T, -1), w4, N, stream=side)
        side.synchronize()
        assert torch.equal(got, want[0])
        inp = x[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q, sc = mxq.mxq_inv_rope_group_quant(inp)
            out = mxq.mxq_linear_a8w4(q.view(T, K), sc.view(T, -1), w4, N)
        for i in (1, 2, 0):
            inp.copy_(x[i])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i])
