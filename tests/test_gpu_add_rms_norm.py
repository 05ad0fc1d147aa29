"""mxq_add_rms_norm: the stored sum bit for bit, the norm within its rounding of the 64-bit value, the codes and
scales bit for bit those of the norm's BF16 output.

Tolerance of y: half a BF16 step, 2^-8 of the value, and the FP32 error before it: the mean of D squares (partial
sums of at most 64 terms a thread and ten levels of pairs: below 2^-17), its root and two products (2^-21):
2^-16 in all."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
import workloads as W
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def inputs(T, D, seed, std=1.0):
    x = W.bf16_normal((T, D), seed=seed, std=std, outlier_frac=0.01).cuda()
    r = W.bf16_normal((T, D), seed=seed + 1, std=2 * std).cuda()
    w = (1 + 0.3 * W.f32_normal((D,), seed=seed + 2)).bfloat16().cuda()
    return x, r, w


def check_y(y, s, w, eps):
    want = ref.norm(s.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), eps)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -133)


def check_codes(q, sc, y):
    codes, scales = O.group_quant_rows(y.float().cpu().numpy())
    assert np.array_equal(sc.cpu().numpy(), scales)
    assert np.array_equal(q.cpu().numpy(), codes)


SIZES = [(1, 16), (3, 32), (5, 128), (9, 144), (33, 256), (17, 272), (16, 512), (7, 528), (8, 1024), (5, 1040), (4, 2048),
         (3, 2064), (1, 4096), (65, 4096), (2, 4112), (3, 8192), (2, 8208), (2, 16384), (2, 16400), (1, 65536), (2, 40000)]


@pytest.mark.parametrize("T,D", SIZES)
def test_all_outputs(mxq, T, D):
    x, r, w = inputs(T, D, seed=100 + D)
    s, y, q, sc = mxq.mxq_add_rms_norm(x, w, 1e-6, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(s.view(torch.int16), (x.float() + r.float()).bfloat16().view(torch.int16))
    check_y(y, s, w, 1e-6)
    check_codes(q, sc, y)


@pytest.mark.parametrize("T,D", [(1, 48), (40, 512), (6, 4096), (2, 9008)])
def test_each_output_alone(mxq, T, D):
    x, r, w = inputs(T, D, seed=900 + D)
    full = mxq.mxq_add_rms_norm(x, w, 1e-5, residual=r)
    s, y, q, sc = mxq.mxq_add_rms_norm(x, w, 1e-5, residual=r, want_y=False)
    assert y is None and torch.equal(s, full[0]) and torch.equal(q, full[2]) and torch.equal(sc, full[3])
    s, y, q, sc = mxq.mxq_add_rms_norm(x, w, 1e-5, residual=r, want_codes=False)
    assert q is None and sc is None and torch.equal(s, full[0]) and torch.equal(y, full[1])
    # Without a residual, of the sum itself.
    s, y, q, sc = mxq.mxq_add_rms_norm(full[0], w, 1e-5)
    assert s is None and torch.equal(y, full[1]) and torch.equal(q, full[2]) and torch.equal(sc, full[3])
    s, y, _, _ = mxq.mxq_add_rms_norm(full[0], None, 1e-5, want_codes=False)
    check_y(y, full[0], None, 1e-5)


@pytest.mark.parametrize("T,D", [(50, 512), (9, 1024), (9, 4096)])
def test_in_place(mxq, T, D):
    x, r, w = inputs(T, D, seed=1300 + D)
    s0, y0, q0, sc0 = mxq.mxq_add_rms_norm(x, w, residual=r)
    for into in ("residual", "x"):
        xx, rr = x.clone(), r.clone()
        a, b = (rr, xx) if into == "residual" else (xx, rr)
        s, y, q, sc = mxq.mxq_add_rms_norm(xx, w, residual=rr, residual_out=a, y=b)
        assert s is a and y is b
        assert torch.equal(s, s0) and torch.equal(y, y0) and torch.equal(q, q0) and torch.equal(sc, sc0)


def test_leading_dimensions(mxq):
    x, _, w = inputs(35, 192, seed=1500)
    flat = mxq.mxq_add_rms_norm(x, w)
    s, y, q, sc = mxq.mxq_add_rms_norm(x.view(7, 5, 192), w)
    assert y.shape == (7, 5, 192) and sc.shape == (7, 5, 2)
    assert torch.equal(y.view(35, 192), flat[1]) and torch.equal(sc.view(35, 2), flat[3])


def test_large_small_and_zero_rows(mxq):
    D = 512
    x = torch.zeros((6, D), dtype=torch.bfloat16, device="cuda")
    x[1] = 1e17          # squares of 1e34: their sum of 5e36 is inside FP32
    x[2] = 1e-30         # squares vanish beside eps
    x[3, 7] = 3.0
    x[4] = -0.0
    x[5, ::2] = 2.0 ** -126
    _, y, q, sc = mxq.mxq_add_rms_norm(x, None, 1e-6)
    check_y(y, x, None, 1e-6)
    check_codes(q, sc, y)


def test_nan_and_infinite_rows_stay_apart(mxq):
    for D in (512, 4096):
        x, _, w = inputs(24, D, seed=1700)
        good = mxq.mxq_add_rms_norm(x, w)
        bad = x.clone()
        bad[3, 5], bad[10, 77], bad[17, D - 1] = float("nan"), float("inf"), -float("inf")
        _, y, q, sc = mxq.mxq_add_rms_norm(bad, w)
        keep = torch.ones(24, dtype=torch.bool)
        keep[[3, 10, 17]] = False
        assert torch.equal(y[keep], good[1][keep]) and torch.equal(q[keep], good[2][keep])
        assert torch.equal(sc[keep], good[3][keep])
        assert bool(torch.isnan(y[3]).all())
        for t, c in ((10, 77), (17, D - 1)):
            assert bool(torch.isnan(y[t, c]))


def test_many_short_rows(mxq):
    """More rows than fit the device at once, and a last CTA of eight rows that is not full."""
    T, D = 100003, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    _, y, q, sc = mxq.mxq_add_rms_norm(x, None)
    v = x.double()
    want = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -16)).all())
    check_codes(q[-50:], sc[-50:], y[-50:])


def test_large_offsets(mxq):
    """Elements past 2^31."""
    T, D = 65537 * 2, 16400
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[-1] = W.bf16_normal((1, D), seed=3).cuda()[0]
    _, y, q, sc = mxq.mxq_add_rms_norm(x, None)
    check_y(y[-1:], x[-1:], None, 1e-6)
    check_codes(q[-1:], sc[-1:], y[-1:])
    assert int(q[:-1].count_nonzero()) == 0 and int(sc[:-1].count_nonzero()) == 0


def test_against_the_two_call_sequence(mxq):
    """The codes are those of the library's quantiser on y."""
    x, r, w = inputs(200, 4096, seed=2100)
    _, y, q, sc = mxq.mxq_add_rms_norm(x, w, residual=r)
    q2, sc2 = mxq.mxq_inv_rope_group_quant(y.view(200, 1, 4096))
    assert torch.equal(q, q2.view(200, 4096)) and torch.equal(sc, sc2.view(200, 32))
