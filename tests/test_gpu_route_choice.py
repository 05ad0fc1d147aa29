"""mxq_route's choice where FP32 scores cannot make it: ids exactly those of the 64-bit reference, weights within 2^-18
(see test_gpu_route.py)."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def cuda(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda()


# Grids of a few logits, all of them BF16 numbers, with one bias for all experts: FP32 scores are equal or next to it,
# 64-bit ones are not.  (least logit, number of steps, step, bias)
CROWDS = {
    "sigmoid": [(16.0, 64, 0.125, 0.0), (16.0, 16, 0.25, 0.5), (-2.0, 32, 0.125, 2.0 ** 17)],
    "softmax": [(0.0, 16, 0.125, 2.0 ** 17), (-3.0, 5, 0.25, 2.0 ** 15)],
    "sqrtsoftplus": [(-3.0, 16, 0.125, 2.0 ** 17), (16.0, 64, 0.125, 2.0 ** 17)],
}


def crowd(scoring, which, T, E, seed):
    """Rows of E logits of that grid, and rows of which only a few lead and the others are far behind."""
    lo, steps, step, bias = CROWDS[scoring][which]
    g = np.random.default_rng(seed)
    l = lo + step * g.integers(0, steps, (T, E))
    few = g.random((T, E)) < np.minimum(1.0, 12.0 / E)
    l[::2] = np.where(few, l, -40.0 if bias < 1 else l - 2.0 ** -6 * E)[::2]
    return l, np.full(E, bias)


@pytest.mark.parametrize("k", [1, 2, 5, 8, 9])
@pytest.mark.parametrize("scoring,which", [(s, i) for s, c in CROWDS.items() for i in range(len(c))])
def test_leaders_that_tie_before_a_larger_one(mxq, scoring, which, k):
    """The k-th and the next pick are the same in logit and bias, and behind them stands one that FP32 does not see to
    be larger."""
    for E, groups in ((12, ()), (24, ((4, 2),)), (64, ((8, 3), (4, 2))), (256, ((8, 4),)), (160, ((8, 3), (5, 2)))):
        l, b = crowd(scoring, which, 12, E, seed=E + 7 * k + which)
        for x in (cuda(l), cuda(l).bfloat16()):
            for kw in (dict(), *(dict(groups=g, topk_groups=t) for g, t in groups)):
                check(mxq, x, cuda(b), k=k, scoring=scoring, **kw)


def test_the_larger_one_comes_last(mxq):
    l = [[17, 17, 17.125, -5], [20, 20, 25, 20], [18, 18, 18, 18.125]]
    check(mxq, cuda(l), cuda([0, 0, 0, 0]), k=1, scoring="sigmoid")
    ids, _ = mxq.mxq_route(cuda(l), 1, scoring="sigmoid", bias=cuda([0, 0, 0, 0]))
    assert ids.flatten().tolist() == [2, 2, 3]
    l = [[-3, -3, -3, -2.99999], [-3, -3, -2.99999, -3]]
    for scoring in ("sigmoid", "softmax", "sqrtsoftplus"):
        for k in (1, 2, 3):
            check(mxq, cuda(l), cuda([8, 8, 8, 8]), k=k, scoring=scoring)


def test_nothing_but_ties(mxq):
    """Rows that indices settle: all alike, fewer kinds than picks, and as many picks as a warp has lanes."""
    for E in (8, 40, 64, 1024):
        l = np.zeros((3, E))
        l[1] = 20.0
        l[2, E // 2:] = 1.0
        for k in (1, 7, 8) + ((31, 32) if E > 32 else ()):
            for scoring in ("sigmoid", "softmax", "sqrtsoftplus"):
                check(mxq, cuda(l), cuda(np.zeros(E)), k=k, scoring=scoring)
    l = np.full((2, 64), 20.0)
    l[0, 63], l[1, 40] = 20.125, 20.5  # ... and with one that is larger
    for k in (1, 8, 31, 32):
        check(mxq, cuda(l), cuda(np.zeros(64)), k=k, scoring="sigmoid")


def test_duplicated_logits_of_a_wide_row(mxq):
    """BF16 logits around 10: sigmoids near 1, with duplicates among the first."""
    g = np.random.default_rng(3)
    l = cuda(10 + 5 * g.standard_normal((400, 256))).bfloat16().clamp_(max=26)
    check(mxq, l, cuda(np.zeros(256)), k=8, scoring="sigmoid")
    check(mxq, l, cuda(np.zeros(256)), undecided=0.01, k=8, scoring="sigmoid", groups=8, topk_groups=4)


@pytest.mark.parametrize("E,groups,keep,top", [(64, 32, 7, 2), (64, 16, 5, 2), (60, 15, 6, 2), (256, 32, 9, 2), (96, 32, 11, 1)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax", "sqrtsoftplus"])
def test_group_values_whose_terms_cancel(mxq, scoring, E, groups, keep, top):
    """Biases of opposite sign leave sums of two that are small beside what they were rounded at."""
    g = np.random.default_rng(E + groups)
    n = E // groups
    for size in (30.0, 1000.0, 2.0 ** 14):
        b = np.full((groups, n), -5.0 * size)
        b[:, 0], b[:, 1] = size, -size
        l = 0.5 + 2.0 ** -10 * g.standard_normal((30, E))
        check(mxq, cuda(l), cuda(b.reshape(-1)), k=6, scoring=scoring, groups=groups, topk_groups=keep, group_top=top)


@pytest.mark.parametrize("E,groups,keep", [(64, 8, 3), (64, 32, 5), (60, 5, 2), (256, 4, 1)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax", "sqrtsoftplus"])
def test_biases_of_the_lowest_value(mxq, scoring, E, groups, keep):
    """Groups whose sum of two is past FP32's range still come before those with nothing to choose, in their order."""
    g = np.random.default_rng(E + groups)
    lowest = torch.finfo(torch.float32).min
    n = E // groups
    l = 1.5 * g.standard_normal((8, E))
    l[:, :n] = -np.inf                              # the first group has nothing
    for seen in ([], [E - 1], [E - n, E // 2], [n + 1]):
        for low in (lowest, -2e38, np.where(np.arange(E) % (2 * n) < n, -3e38, -2.5e38)):
            b = np.full(E, 1.0) * low
            b[seen] = 0.1
            # (Such a bias is the sum in any arithmetic, so that 64 bits decide every row: ties go by index.)
            kw = dict(k=4, scoring=scoring, groups=groups, topk_groups=keep)
            ids, _ = mxq.mxq_route(cuda(l), bias=cuda(b), **kw)
            want, _, _ = ref.route(cuda(l).double().cpu().numpy(), bias=cuda(b).double().cpu().numpy(), **kw)
            assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:5]


@pytest.mark.parametrize("renormalise", [False, True])
def test_weights_of_very_negative_logits(mxq, renormalise):
    """sqrt(log(1 + exp(l))) is about exp(l / 2): inside FP32's range where exp(l) is not."""
    l = np.stack([np.linspace(-170, -100, 64), np.linspace(-120, -80, 64), np.linspace(-40, 10, 64), np.linspace(-17, -15, 64)])
    for bias in (None, cuda(np.zeros(64))):
        check(mxq, cuda(l), bias, k=12, scoring="sqrtsoftplus", renormalise=renormalise)
        check(mxq, cuda(l[:, ::-1].copy()), bias, k=12, scoring="sqrtsoftplus", renormalise=renormalise, groups=8, topk_groups=3)
    for at in range(0, 64, 8):
        check(mxq, cuda(l[:, at:at + 8]), None, k=8, scoring="sqrtsoftplus", renormalise=renormalise)


@pytest.mark.parametrize("renormalise", [False, True])
def test_weights_far_from_the_largest_logit(mxq, renormalise):
    """exp(l - max) where the difference itself is rounded: by 2^-18 at 64 and more."""
    g = np.random.default_rng(8)
    l = np.concatenate([-60 * g.random((200, 32)), -84 * g.random((800, 32))]) + 7 * g.random((1000, 1))
    for bias in (None, cuda(np.zeros(32))):
        check(mxq, cuda(l), bias, k=32, scoring="softmax", renormalise=renormalise)
