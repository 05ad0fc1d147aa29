"""mxq_rope_kv4_insert and mxq_kv4_gather bit for bit against the 64-bit
reference: query bits, codes, scale bytes, rows not addressed, data errors."""

import numpy as np
import pytest
import torch

import attn_ref as ref
import workloads as W
from cases import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def inputs(T, H, Dq, Dk, R, seed, max_pos=5000, kv_std=4.0):
    q = W.bf16_normal((T, H, Dq), seed=seed)
    kv = W.bf16_normal((T, Dk), seed=seed + 1, std=kv_std, outlier_frac=0.01)
    pos = W.positions_uniform(T, seed=seed + 2, max_pos=max_pos)
    cos, sin = W.rope_cache(max_pos, max(R, 2))
    slots = np.random.Generator(np.random.PCG64(seed + 3)).permutation(2 * T + 3)[:T].astype(np.int64)
    return q, kv, pos, cos, sin, slots, 2 * T + 3


def run(mxq, q, kv, pos, cos, sin, R, slots, ns, inplace=False):
    Dk = kv.shape[1]
    qd, kvd, pd, cd, sd = to_dev(q, kv, pos, cos, sin)
    cache = torch.full((ns, Dk // 2), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((ns, Dk // 32), 0x5A, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mxq.mxq_rope_kv4_insert(qd, kvd, pd, cd, sd, R, torch.from_numpy(slots).cuda(), cache, sf,
                                  q_out=qd if inplace else None, err_flag=err)
    torch.cuda.synchronize()
    return out, cache.cpu().numpy(), sf.cpu().numpy(), int(err.item())


def want(q, kv, pos, cos, sin, R, slots, ns):
    Dk = kv.shape[1]
    cache, sf = np.full((ns, Dk // 2), 0xA5, np.uint8), np.full((ns, Dk // 32), 0x5A, np.uint8)
    c, s = cos.double().numpy()[pos.numpy()], sin.double().numpy()[pos.numpy()]
    qr, y = q.float().numpy(), kv.float().numpy()
    if R:
        qr, y = ref.rotate(qr, c, s, R), ref.rotate(y, c, s, R)
    codes, bytes_ = ref.encode_e2m1(y)
    ok = slots >= 0
    cache[slots[ok]], sf[slots[ok]] = codes[ok], bytes_[ok]
    return W.bf16_bits(torch.from_numpy(qr).bfloat16()), cache, sf


@pytest.mark.parametrize("T,H,Dq,Dk,R", [(1, 64, 512, 512, 64), (64, 64, 512, 512, 64), (37, 3, 192, 576, 16),
                                         (37, 3, 192, 576, 48), (33, 2, 128, 128, 128), (5, 1, 64, 32, 0),
                                         (200, 16, 256, 96, 32)])
def test_bits(mxq, T, H, Dq, Dk, R):
    a = inputs(T, H, Dq, Dk, R, seed=7000 + T)
    out, cache, sf, err = run(mxq, *a[:5], R, *a[5:])
    q, c, s = want(*a[:5], R, *a[5:])
    assert err == 0
    assert np.array_equal(W.bf16_bits(out.cpu()), q)
    assert np.array_equal(sf, s) and np.array_equal(cache, c)


def test_in_place_and_padding_slots(mxq):
    a = list(inputs(50, 8, 256, 256, 64, seed=7100))
    a[5][::3] = -1
    out, cache, sf, err = run(mxq, *a[:5], 64, *a[5:], inplace=True)
    q, c, s = want(*a[:5], 64, *a[5:])
    assert err == 0 and np.array_equal(W.bf16_bits(out.cpu()), q)
    assert np.array_equal(sf, s) and np.array_equal(cache, c)


def test_streamed_query(mxq):
    """A query of 32 MiB or more goes through the streaming copy; the KV rows as ever."""
    a = inputs(2000, 16, 576, 576, 64, seed=7200)
    out, cache, sf, err = run(mxq, *a[:5], 64, *a[5:])
    q, c, s = want(*a[:5], 64, *a[5:])
    assert err == 0 and np.array_equal(W.bf16_bits(out.cpu()), q)
    assert np.array_equal(sf, s) and np.array_equal(cache, c)


def test_ties_ranges_and_zeros(mxq):
    """Every tie of the encoding, blocks of zeros, of the smallest and the largest BF16 values, amax at and
    just above 6 * 2^e, negative zeros."""
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0,
                     -0.0], np.float32)
    for e in (-100, -3, 0, 1, 60, 120):
        rows.append(np.concatenate([ties, ties]) * np.float32(2.0 ** e))
    rows.append(np.zeros(32, np.float32))
    rows.append(np.full(32, 2.0 ** -133, np.float32))
    rows.append(np.full(32, 2.0 ** -126, np.float32))
    rows.append(np.full(32, 3.3895e38, np.float32))
    rows.append(np.linspace(-6.03125, 6.03125, 32).astype(np.float32))
    kv = torch.from_numpy(np.stack(rows)).bfloat16()
    T = kv.shape[0]
    q, _, pos, cos, sin, slots, ns = inputs(T, 1, 64, 32, 0, seed=7300)
    _, cache, sf, err = run(mxq, q, kv, pos, cos, sin, 0, slots, ns)
    _, c, s = want(q, kv, pos, cos, sin, 0, slots, ns)
    assert err == 0 and np.array_equal(sf, s)
    assert np.array_equal(cache, c)


def test_non_finite_blocks(mxq):
    q, kv, pos, cos, sin, slots, ns = inputs(4, 1, 64, 128, 0, seed=7400)
    kv[0, 5], kv[1, 40], kv[2, 127] = float("nan"), float("inf"), float("-inf")
    _, _, sf, _ = run(mxq, q, kv, pos, cos, sin, 0, slots, ns)
    got = sf[slots] == 255
    assert got.tolist() == [[True, False, False, False], [False, True, False, False],
                            [False, False, False, True], [False] * 4]


def test_invalid_positions_and_slots(mxq):
    q, kv, pos, cos, sin, slots, ns = inputs(12, 4, 256, 256, 64, seed=7500, max_pos=100)
    pos[[2, 7]] = torch.tensor([100, -3])
    slots[5] = ns
    out, cache, sf, err = run(mxq, q, kv, pos, cos, sin, 64, slots, ns)
    assert err == mxq.MXQ_DEVERR_POSITION | mxq.MXQ_DEVERR_SLOT
    good = np.array([t for t in range(12) if t not in (2, 7)])
    gs = slots[good].copy()
    gs[gs >= ns] = -1
    wq, c, s = want(q[good], kv[good], pos[good], cos, sin, 64, gs, ns)
    got = W.bf16_bits(out.cpu())
    assert np.array_equal(got[good], wq) and (got[[2, 7], :, 192:] == 0).all()
    assert np.array_equal(cache, c) and np.array_equal(sf, s)


def test_gather(mxq):
    """All 16 codes under every scale byte, as BF16; slots outside the cache."""
    codes = torch.from_numpy(np.tile(np.arange(256, dtype=np.uint8), (256, 1))).cuda()
    sf = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 16).contiguous()
    slots = torch.tensor([*range(255, -1, -1), -1, 256], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mxq.mxq_kv4_gather(codes, sf, slots, err_flag=err).cpu()
    with np.errstate(over="ignore"):
        v = ref.e2m1_values(codes.cpu().numpy(), sf.cpu().numpy())[::-1].copy()
    w = torch.from_numpy(v).bfloat16()
    assert torch.equal(torch.isnan(out[:256]), torch.isnan(w))
    ok = ~torch.isnan(w)
    assert torch.equal(out[:256][ok].view(torch.int16), w[ok].view(torch.int16))
    assert (out[256:].float() == 0).all() and int(err.item()) == mxq.MXQ_DEVERR_SLOT


def test_binding_refuses(mxq):
    q, kv, pos, cos, sin, slots, ns = inputs(4, 2, 128, 128, 64, seed=7600)
    d = to_dev(q, kv, pos, cos, sin)
    sl = torch.from_numpy(slots).cuda()
    cache = torch.zeros((ns, 64), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((ns, 4), dtype=torch.uint8, device="cuda")
    good = dict(q=d[0], kv=d[1], pos=d[2], cos=d[3], sin=d[4], R=64, slot_mapping=sl, cache=cache, cache_sf=sf)
    mxq.mxq_rope_kv4_insert(**good)
    for bad in (dict(q=d[0].float()), dict(kv=d[1].float()), dict(kv=d[1][:, ::2]), dict(slot_mapping=sl.int()),
                dict(cache=cache[:, :32]), dict(cache_sf=sf[:, :2]), dict(cache_sf=sf[:-1]), dict(R=24),
                dict(pos=d[2].int()), dict(cos=d[3].float())):
        with pytest.raises(mxq.MxqError):
            mxq.mxq_rope_kv4_insert(**{**good, **bad})
    for bad in (dict(slots=sl.int()), dict(cache_sf=sf[:, :2]), dict(cache=cache.float())):
        with pytest.raises(mxq.MxqError):
            mxq.mxq_kv4_gather(**{**dict(cache=cache, cache_sf=sf, slots=sl), **bad})
