"""mxq_experts_a8w4: the results that a token's experts add to its sum are FP32, in calls of any size.  The tolerance is
that of ffn_ref.experts without its term for results held to a share of their neighbours: 1e-5 of each product's
magnitudes for the FP32 sums, what these can move the 8-bit codes in between, and half a BF16 step of the result."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
from test_gpu_experts import Layer, choose, unit_acts
from test_gpu_w4 import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def expected(a, ids, wt, w13, w2):
    """-> (64-bit results, tolerance) of ffn_ref.experts' arguments."""
    T, N = a.shape[0], w2.shape[1]
    out, tol = np.zeros((T, N)), np.zeros((T, N))
    for e in range(w2.shape[0]):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        g, sg = ref.linear(a[t], w13[e, 0])
        u, su = ref.linear(a[t], w13[e, 1])
        silu = g / (1 + np.exp(-g))
        h = silu * u
        err = 1.1 * np.abs(u) * 1e-5 * sg + np.abs(silu) * 1e-5 * su + (2.0 ** -20 + 2.0 ** -22 * np.abs(g)) * np.abs(h)
        q, slack = ref.quant_with_slack(h, err)
        y, sy = ref.linear(q, w2[e])
        w = wt[t, j][:, None]
        np.add.at(out, t, w * y)
        np.add.at(tol, t, np.abs(w) * (1e-5 * sy + slack @ np.abs(w2[e]).T))
    return out, tol + np.abs(out) * 2.0 ** -8 + 2.0 ** -126


class Outliers(Layer):
    """A layer in which one column of each 32 of the result is 2^`up` times larger than the others."""

    def __init__(self, mxq, E, K, I, N, seed, up):
        super().__init__(mxq, E, K, I, N, seed)
        codes, sf = self.w2
        sf[:, 5::32] += up
        self.p2 = mxq.mxq_prepare_w4(*dev(codes, sf))


@pytest.mark.parametrize("up", [0, 5, 7])
@pytest.mark.parametrize("T,k,E,K,I,N", [(4, 4, 8, 256, 128, 272), (40, 3, 40, 256, 128, 272), (60, 4, 12, 256, 128, 304),
                                         (130, 4, 8, 128, 96, 528), (400, 4, 8, 128, 96, 528), (90, 12, 8, 128, 64, 80)])
def test_small_columns_beside_large_ones(mxq, T, k, E, K, I, N, up):
    layer = Outliers(mxq, E, K, I, N, seed=T, up=up)
    a, asf = unit_acts(T, K, seed=T + 1)
    ids, wt = choose(T, min(k, E), E, seed=T + 2)
    out = layer(a, asf, ids, wt)
    want, tol = expected(ref.act_values(a, asf), ids, wt.astype(np.float64), *layer.values())
    bad = ~(np.abs(out.double().cpu().numpy() - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


def test_large_weights_of_zero_results(mxq):
    """A result of zero stays zero beside large ones and under a large weight."""
    T, E = 200, 3
    layer = Layer(mxq, E, 128, 64, 64, seed=50)
    codes, sf = layer.w2
    codes[:, 1::2] = 0
    sf[:, ::2] = 210
    layer.p2 = mxq.mxq_prepare_w4(*dev(codes, sf))
    a, asf = unit_acts(T, 128, seed=51)
    ids, wt = choose(T, 2, E, seed=52)
    out = layer(a, asf, ids, np.full_like(wt, 2.0 ** 60))
    assert int(out[:, 1::2].count_nonzero()) == 0
