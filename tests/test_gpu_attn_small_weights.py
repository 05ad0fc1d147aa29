"""mxq_attn where one key leads its row by far and the columns it holds zeros in
are made up by thousands of keys of small weight: what a first key that draws
most of the attention looks like.

The scores are a staircase over the heads: head h's leading key is 0.45 (h + 1)
octaves (factors of two in the weight) above the others.  The leading key holds
zeros from column 2 on, the others values of mean 1, so that an error which all
small weights share shows undiminished.

Tolerances.  A weight is rounded to BF16 or better (2^-8 of itself at most), the
output once more (2^-8): 2^-7 of A = sum_j w_j |k_j|.  Scores are off by 2^-19 of
sabs = sm_scale * sum_d |q_d k_d| at most, which moves a weight and the
denominator by as much.  E4M3 rows: a weight below 2^-22 of the largest is off by
2^-30 of the largest at most instead.
"""

import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu

SCALE8 = 2.0 ** -4


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def stored(cache, x):
    """x float32 [n, D] -> (cache tensor, cache_sf, kv_scale, the 64-bit values the cache stands for)."""
    if cache == "bf16":
        kv = torch.from_numpy(x).bfloat16()
        return kv, None, None, kv.double().numpy()
    if cache == "e4m3":
        kv = (torch.from_numpy(x) / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return kv, None, SCALE8, ref.e4m3_values(kv.numpy()) * SCALE8
    codes, sf = ref.encode_e2m1(x)
    return torch.from_numpy(codes), torch.from_numpy(sf), None, ref.e2m1_values(codes, sf)


def attend(mxq, q, kv, sf, scale, bt, lens, page, **kw):
    d = "cuda"
    lse = torch.empty(q.shape[:2], device=d)
    out = mxq.mxq_attn(q.to(d), kv.to(d), torch.from_numpy(bt).to(d), torch.tensor(lens, dtype=torch.int32, device=d),
                       page_size=page, lse=lse, cache_sf=None if sf is None else sf.to(d),
                       kv_scale=None if scale is None else torch.tensor([scale], device=d), **kw)
    torch.cuda.synchronize()
    assert mxq.mxq_watchdog_read() == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def check(cache, got, lse, want, rows):
    o, l, A, sabs = want
    ds = 2.0 ** -19 * sabs
    # No weight exceeds 1, the denominator is 1 or more in units of the largest.
    low = rows.shape[0] * 2.0 ** -30 * np.abs(rows).max() if cache == "e4m3" else 0.0
    tol = A * (2.0 ** -7 + 2 * ds[..., None]) + low + 1e-30
    assert np.isfinite(got).all()
    worst = np.abs(got - o) / tol
    assert worst.max() <= 1.0, f"{worst.max():.2f} of the tolerance, head {np.unravel_index(worst.argmax(), worst.shape)[1]}"
    # 2^-22 relative, 2^-17 for the logarithm and the sum of rounded exponentials.
    assert (np.abs(lse - l) <= ds + 2.0 ** -22 * np.abs(l) + 2.0 ** -17).all()


def staircase(cache, H, D, n, lead, spread, seed):
    """q [1, H, D] and n keys of which number `lead` leads; spread: the others differ by up to an octave."""
    rng = np.random.Generator(np.random.PCG64(seed))
    x = np.zeros((n, D), np.float32)
    # Powers of two and eighths: E4M3 and BF16 hold them, and E2M1 something close, which the reference reads back.
    x[:, 2:] = rng.choice([0.5, 0.75, 1.0, 1.25, 1.5], (n, D - 2))
    if spread:
        x[:, 1] = rng.choice([0.0, 0.25, 0.5, 0.75, 1.0], n)
    x[lead] = 0.0
    x[lead, 0] = 24.0
    kv, sf, scale, rows = stored(cache, x)
    q = np.zeros((1, H, D), np.float32)
    q[0, :, 0] = 0.45 * (np.arange(H) % 64 + 1) * np.log(2.0) / rows[lead, 0]
    q[0, :, 1] = np.log(2.0)
    return torch.from_numpy(q).bfloat16(), kv, sf, scale, rows


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("H,D,n", [(64, 128, 9000), (64, 512, 5000), (20, 192, 3000), (128, 64, 20000)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("spread", [False, True])
def test_one_leading_key(mxq, cache, H, D, n, where, spread):
    """One sequence, its keys split over many CTAs and joined."""
    lead = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[where]
    page = 48
    pages = -(-n // page)
    q, kv, sf, scale, rows = staircase(cache, H, D, pages * page, lead, spread, seed=n + H)
    bt = np.arange(pages, dtype=np.int32)[None]
    got, lse = attend(mxq, q, kv, sf, scale, bt, [n], page, sm_scale=1.0)
    want = ref.attention(q.double().numpy(), rows, bt, page, np.array([0, 1]), [n], 0, 0, 1.0)
    check(cache, got, lse, want, rows)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("where", ["first", "last"])
def test_one_leading_key_whole_tiles(mxq, cache, where):
    """304 sequences of 8192 keys (the same pages), two tiles a CTA: every tile is walked by one CTA.  All
    sequences have the same bits, and the first agrees with the reference."""
    H, D, n, B, page = 64, 128, 8192, 304, 64
    q, kv, sf, scale, rows = staircase(cache, H, D, n, 0 if where == "first" else n - 1, True, seed=77)
    bt = np.arange(n // page, dtype=np.int32)[None]
    got, lse = attend(mxq, q.expand(B, -1, -1).contiguous(), kv, sf, scale, np.repeat(bt, B, 0), [n] * B, page,
                      sm_scale=1.0)
    assert (got == got[:1]).all() and (lse == lse[:1]).all()
    want = ref.attention(q.double().numpy(), rows, bt, page, np.array([0, 1]), [n], 0, 0, 1.0)
    check(cache, got[:1], lse[:1], want, rows)


@pytest.mark.parametrize("H", [16, 64])
def test_zeros_under_the_largest_weights_e4m3(mxq, H):
    """Most columns of the keys with the largest scores hold zeros, so that keys of small weight, in later
    blocks too, make up the output there."""
    D, n, page = 128, 1024, 64
    rng = np.random.Generator(np.random.PCG64(60))
    x = (rng.standard_normal((n, D)) * 3.0).astype(np.float32)
    x[rng.random((n, D)) < 0.6] = 0.0
    kv, sf, scale, rows = stored("e4m3", x)
    q = (torch.randn((9, H, D), generator=torch.Generator().manual_seed(61)) * 2.0).bfloat16()
    bt = rng.permutation(n // page).astype(np.int32)[None]
    start = np.array([0, 9], np.int32)
    got, lse = attend(mxq, q, kv, sf, scale, bt, [900], page, q_start=torch.from_numpy(start).cuda())
    want = ref.attention(q.double().numpy(), rows, bt, page, start, [900], 0, 0, D ** -0.5)
    check("e4m3", got, lse, want, rows)
