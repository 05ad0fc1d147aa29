"""mxq_attn over what a cache can hold and how a batch can look: scale bytes of
the 4-bit cache far from 127 and at its ends, every finite E4M3 code, weights
of very different sizes on columns that mostly hold zeros, and drawn batches.

Tolerances.  A weight below 1/16 of its row's sum is rounded to BF16 or better
(half an ulp: 2^-8 of itself at most), the output once more: with
A = sum_j w_j |k_j| >= |out| the two stay within 2^-7 * A.  The scores, FP32 sums
of D exact products, are off by 2^-19 of sabs = sm_scale * sum_d |q_d k_d| at
most, which moves a weight and the denominator by as much.  Weights below 2^-26
of the largest may count as zero (E4M3): 2^-20 of the largest key per 64 of them.
"""

import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def run_and_check(mxq, q, cache, sf, scale8, rows, lens, nq, page, window=0, sinks=0, seed=0):
    """q bf16 [T, H, D]; the keys of all sequences lie in shuffled pages of `rows` (64-bit values)."""
    T, H, D = q.shape
    B, d = len(lens), "cuda"
    pages = max(1, -(-max(lens) // page))
    rng = np.random.Generator(np.random.PCG64(seed))
    bt = rng.permutation(rows.shape[0] // page)[:B * pages].astype(np.int32).reshape(B, pages)
    start = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    lse = torch.empty((T, H), device=d)
    err = torch.zeros(1, dtype=torch.int32, device=d)
    out = mxq.mxq_attn(q.to(d), cache.to(d), torch.from_numpy(bt).to(d), torch.tensor(lens, dtype=torch.int32, device=d),
                       q_start=torch.from_numpy(start).to(d), page_size=page, window=window, sinks=sinks,
                       kv_scale=None if scale8 is None else torch.tensor([scale8], device=d),
                       cache_sf=None if sf is None else sf.to(d), lse=lse, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and mxq.mxq_watchdog_read() == 0
    o, l, A, sabs = ref.attention(q.double().numpy(), rows, bt, page, start, lens, window, sinks, D ** -0.5)
    ds = 2.0 ** -19 * sabs
    low = 0.0 if scale8 is None else 2.0 ** -26 * max(lens) * np.abs(rows).max()
    tol = A * (2.0 ** -7 + 2 * ds[..., None]) + low + 1e-37
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - o) / tol).max() <= 1.0
    g, empty = lse.double().cpu().numpy(), np.isinf(l)
    assert np.array_equal(np.isneginf(g), empty)
    # 2^-22 relative, 2^-17 for the logarithm and the sum of rounded exponentials.
    assert (np.abs(g[~empty] - l[~empty]) <= ds[~empty] + 2.0 ** -22 * np.abs(l[~empty]) + 2.0 ** -17).all()


@pytest.mark.parametrize("H", [1, 20, 64])
def test_e2m1_scale_bytes(mxq, H):
    """Blocks of 32 columns with scales from 2^-100 to 2^53 next to each other, the query scaled against them;
    the columns of byte 0 (2^-127, below BF16's normal range) have no query."""
    bytes_ = np.array([27, 60, 100, 126, 127, 128, 129, 140, 180, 0])
    D, n, rng = 32 * len(bytes_), 640, np.random.Generator(np.random.PCG64(40 + H))
    codes = rng.integers(0, 256, (n, D // 2)).astype(np.uint8)
    sf = np.broadcast_to((bytes_ + rng.integers(0, 2, (n, len(bytes_)))), (n, len(bytes_))).astype(np.uint8)
    rows = ref.e2m1_values(codes, sf)
    down = np.repeat(np.where(bytes_ == 0, 0.0, 2.0 ** (127.0 - bytes_)), 32)
    q = (torch.randn((3, H, D), generator=torch.Generator().manual_seed(H)).double() * torch.from_numpy(down)).bfloat16()
    run_and_check(mxq, q, torch.from_numpy(codes), torch.from_numpy(sf), None, rows, [300, 129], [2, 1], 16)


@pytest.mark.parametrize("H,D", [(16, 192), (64, 512)])
def test_e4m3_every_code(mxq, H, D):
    """All finite codes, subnormals and zeros among them, equally often."""
    rng = np.random.Generator(np.random.PCG64(50))
    codes = rng.integers(0, 254, (1056, D))
    codes = (codes + (codes >= 127)).astype(np.uint8)  # without 0x7F and 0xFF
    scale = np.float32(0.013)
    q = (torch.randn((5, H, D), generator=torch.Generator().manual_seed(51)) * 0.1).bfloat16()
    run_and_check(mxq, q, torch.from_numpy(codes), None, float(scale), ref.e4m3_values(codes) * np.float64(scale),
                  [500, 130], [1, 4], 32)


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
def test_zeros_under_the_largest_weights(mxq, cache):
    """Most columns of the keys with the largest scores hold zeros, so that keys of small weight, in later
    blocks too, make up the output there."""
    D, H, n = 128, 16, 1024
    rng = np.random.Generator(np.random.PCG64(60))
    x = rng.standard_normal((n, D)) * 3.0
    x[rng.random((n, D)) < 0.6] = 0.0
    if cache == "bf16":
        kv, sf = torch.from_numpy(x).bfloat16(), None
        rows = kv.double().numpy()
    else:
        codes, s = ref.encode_e2m1(x.astype(np.float32))
        kv, sf, rows = torch.from_numpy(codes), torch.from_numpy(s), ref.e2m1_values(codes, s)
    q = (torch.randn((9, H, D), generator=torch.Generator().manual_seed(61)) * 2.0).bfloat16()
    run_and_check(mxq, q, kv, sf, None, rows, [900], [9], 64)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(mxq, seed):
    """Batches drawn over the argument ranges: heads, columns, pages, lengths of zero up, chunks, windows."""
    rng = np.random.Generator(np.random.PCG64(700 + seed))
    cache = ["bf16", "e4m3", "e2m1"][seed % 3]
    H, D, page = int(rng.integers(1, 97)), 64 * int(rng.integers(1, 9)), 16 * int(rng.integers(1, 9))
    B = int(rng.integers(1, 6))
    nq = [int(rng.choice([0, 1, 1, 2, 7, 40])) for _ in range(B)]
    if sum(nq) == 0:
        nq[0] = 1
    lens = [n + int(rng.choice([0, 1, 15, 130, 600])) for n in nq]
    window = int(rng.choice([0, 0, 1, 50, 128, 500]))
    sinks = int(rng.choice([0, 4, 33])) if window else 0
    n = (B * max(1, -(-max(lens) // page)) + 2) * page
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, D), generator=g)
    sf = scale = None
    if cache == "bf16":
        kv = x.bfloat16()
        rows = kv.double().numpy()
    elif cache == "e4m3":
        scale = float(np.float32(0.02))
        kv = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        rows = ref.e4m3_values(kv.numpy()) * scale
    else:
        codes, s = ref.encode_e2m1(x.numpy())
        kv, sf, rows = torch.from_numpy(codes), torch.from_numpy(s), ref.e2m1_values(codes, s)
    q = torch.randn((sum(nq), H, D), generator=g).bfloat16()
    run_and_check(mxq, q, kv, sf, scale, rows, lens, nq, page, window, sinks, seed)
