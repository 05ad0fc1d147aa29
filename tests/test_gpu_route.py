"""mxq_route: ids exactly those of the 64-bit reference, weights within FP32's rounding of it (exponentials,
sums of up to 1024 terms and two quotients: below 2^-18 of the value)."""

import numpy as np
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def check(mxq, logits, bias=None, undecided=0.0, **kw):
    """`undecided`: the share of rows that 64-bit scores may leave open (see ffn_ref.route)."""
    b = None if bias is None else bias.double().cpu().numpy()
    ids, w = mxq.mxq_route(logits, bias=bias, **kw)
    torch.cuda.synchronize()
    want, ww, sure = ref.route(logits.double().cpu().numpy(), bias=b, **kw)
    assert np.mean(~sure) <= undecided
    ids, w, want, ww = ids.cpu().numpy()[sure], w.double().cpu().numpy()[sure], want[sure], ww[sure]
    assert np.array_equal(ids, want), np.argwhere(ids != want)[:5]
    assert np.all(np.abs(w - ww) <= 2.0 ** -18 * np.abs(ww) + 2.0 ** -126)


def draw(T, E, seed, std=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, E), generator=g, device="cuda") * std, torch.randn((E,), generator=g, device="cuda") * 0.1


CASES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (5, 32, 4, 4, 2), (70, 33, 5, 1, 1), (9, 60, 6, 5, 3), (9, 60, 6, 1, 1),
         (33, 64, 8, 8, 1), (130, 256, 8, 8, 4), (3, 200, 7, 8, 3), (21, 257, 9, 1, 1), (10, 384, 8, 6, 5),
         (4, 512, 32, 16, 9), (3, 1024, 32, 32, 11), (3, 1000, 10, 1, 1), (2, 96, 32, 32, 32), (6, 96, 3, 32, 7)]


@pytest.mark.parametrize("T,E,k,groups,keep", CASES)
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax", "sqrtsoftplus"])
@pytest.mark.parametrize("biased", [False, True])
def test_against_reference(mxq, T, E, k, groups, keep, scoring, biased):
    l, b = draw(T, E, seed=E + k)
    for x in (l, l.bfloat16()):  # BF16 logits tie often
        check(mxq, x, b if biased else None, k=k, scoring=scoring, groups=groups, topk_groups=keep, scale=2.5)


@pytest.mark.parametrize("kw", [dict(renormalise=False), dict(group_top=1, groups=8, topk_groups=3), dict(scale=-0.5),
                                dict(group_top=1, groups=8, topk_groups=8, renormalise=False, scale=16.0)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax", "sqrtsoftplus"])
def test_options(mxq, kw, scoring):
    l, b = draw(50, 64, seed=77)
    for bias in (None, b):
        check(mxq, l, bias, k=6, scoring=scoring, **kw)


def test_near_ties_follow_64_bits(mxq):
    """Rows whose scores differ by less than FP32 resolves, and rows whose scores and biases cross over."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    T, E = 300, 128
    base = torch.randn((T, 1), generator=g, device="cuda")
    step = torch.randint(-6, 7, (T, E), generator=g, device="cuda", dtype=torch.int32)
    l = (base.view(torch.int32) + step).view(torch.float32)  # a few FP32 steps apart
    b = torch.full((E,), 0.25, device="cuda")
    b[::3] += 2.0 ** -23
    for scoring in ("sigmoid", "softmax", "sqrtsoftplus"):
        for kw in (dict(), dict(groups=8, topk_groups=3), dict(groups=16, topk_groups=5, group_top=1)):
            # Sums of two scores whose logits are a few FP32 steps d apart on either side of the same mean
            # differ by d^2 times the score's curvature, 1e-15 and less: 64-bit scores do not tell them apart.
            pairs = kw.get("groups") == 8
            check(mxq, l, b, undecided=0.5 if pairs else 0.0, k=8, scoring=scoring, **kw)
            check(mxq, l, None, undecided=0.5 if pairs else 0.0, k=8, scoring=scoring, **kw)


def test_ties_go_to_the_lowest_index(mxq):
    for E, G in ((256, 8), (60, 5), (1024, 32)):
        l = torch.zeros((3, E), device="cuda")
        l[1, E // 2:] = 1.0
        l[2, ::2] = -0.0
        b = torch.zeros((E,), device="cuda")
        for bias in (None, b):
            for keep in (G, 2):
                check(mxq, l, bias, k=7, scoring="sigmoid", groups=G, topk_groups=keep)


def test_saturated_and_tiny_scores(mxq):
    """Sigmoids of large logits differ by less than FP32 shows, those of very small ones vanish in FP32."""
    E = 64
    l = torch.linspace(-95, -85, E, device="cuda").repeat(4, 1)
    l[1] = torch.linspace(12, 30, E, device="cuda")
    l[2] = torch.linspace(-200, -100, E, device="cuda")
    l[3, ::2] += 100
    b = torch.zeros((E,), device="cuda")
    for scoring in ("sigmoid", "softmax", "sqrtsoftplus"):
        ids, _ = mxq.mxq_route(l, 8, scoring=scoring, bias=b)
        want, _, _ = ref.route(l.double().cpu().numpy(), 8, scoring, bias=b.double().cpu().numpy())
        assert np.array_equal(ids.cpu().numpy(), want)


def test_masked_experts(mxq):
    E, k = 64, 6
    l, b = draw(12, E, seed=5)
    inf = float("inf")
    l[0] = -inf                       # nothing left
    l[1, 3:] = -inf                   # fewer than k
    l[2, ::2] = float("nan")
    l[3] = float("nan")
    l[4] = torch.finfo(torch.float32).min
    l[5] = torch.finfo(torch.float32).min
    l[5, 7] = 0.5
    l[6, 9] = inf
    l[7, 9], l[7, 10] = inf, inf
    l[8, 32:] = -inf
    l[9, 1:8] = -inf                  # one expert left in the first group
    b[20], b[21], b[22] = -inf, float("nan"), inf
    for scoring in ("sigmoid", "softmax"):
        for bias in (None, b):
            for kw in (dict(), dict(groups=8, topk_groups=2), dict(groups=8, topk_groups=2, group_top=1)):
                check(mxq, l, bias, k=k, scoring=scoring, **kw)


def test_unaligned_rows_and_given_outputs(mxq):
    l, b = draw(7, 51, seed=9)
    ids = torch.full((9, 4), -7, dtype=torch.int32, device="cuda")
    w = torch.full((9, 4), -7.0, device="cuda")
    mxq.mxq_route(l, 4, scoring="sigmoid", bias=b, ids=ids[1:8], weights=w[1:8])
    a, c = mxq.mxq_route(l, 4, scoring="sigmoid", bias=b)
    assert torch.equal(ids[1:8], a) and torch.equal(w[1:8], c)
    assert bool((ids[[0, 8]] == -7).all()) and bool((w[[0, 8]] == -7).all())  # rows beside them stay


def test_many_tokens(mxq):
    l, b = draw(20000, 256, seed=10)
    ids, w = mxq.mxq_route(l, 8, scoring="sigmoid", bias=b, groups=8, topk_groups=4)
    p = torch.sigmoid(l.double())
    c = (p + b.double()).view(-1, 8, 32)
    top = c.topk(2, -1).values.sum(-1).topk(4, -1).indices
    see = torch.zeros((20000, 8), dtype=torch.bool, device="cuda").scatter_(1, top, True)
    c = c.masked_fill(~see[..., None], -1e9).view(-1, 256)
    want = c.topk(8, -1).indices
    assert torch.equal(ids.long(), want)
    wp = p.gather(1, want)
    wp = wp / wp.sum(1, keepdim=True)
    assert bool(((w.double() - wp).abs() <= 2.0 ** -18 * wp).all())


@pytest.mark.parametrize("E", [128, 256, 512, 1024])
def test_bias_that_begins_at_any_element(mxq, E):
    l, b = draw(6, E, seed=E)
    want = mxq.mxq_route(l, 5, scoring="sigmoid", bias=b, groups=8, topk_groups=3)
    for at in (1, 2, 3):
        room = torch.full((E + 8,), float("nan"), device="cuda")
        room[at:at + E] = b
        got = mxq.mxq_route(l, 5, scoring="sigmoid", bias=room[at:at + E], groups=8, topk_groups=3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,E,k,groups,keep", [(40, 160, 6, 8, 3), (30, 144, 8, 16, 5), (30, 352, 7, 1, 1), (30, 384, 8, 8, 4),
                                               (30, 768, 12, 2, 1), (25, 40, 4, 4, 2), (25, 72, 5, 8, 2), (25, 1024, 9, 4, 1),
                                               (25, 192, 6, 32, 9), (25, 320, 6, 16, 16), (30, 20, 3, 4, 2)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_uneven_lanes(mxq, T, E, k, groups, keep, scoring):
    """Groups that do not fill their lanes, and lanes of up to 12 experts."""
    l, b = draw(T, E, seed=E + groups)
    for x in (l, l.bfloat16()):
        for bias in (None, b):
            check(mxq, x, bias, k=k, scoring=scoring, groups=groups, topk_groups=keep)
    room = torch.zeros((E + 1,), device="cuda")
    room[1:] = b
    got, want = (mxq.mxq_route(l, k, scoring, bias=v, groups=groups, topk_groups=keep) for v in (room[1:], b))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
