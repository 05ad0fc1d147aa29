"""mxq_experts_a8w4 against the 64-bit definition.  The tolerance (ffn_ref.experts) counts half a BF16 step, 1e-5 of
each product's magnitudes for the FP32 sums, and, where these can carry a value between the products over a rounding
border, one step of its 8-bit code."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
from test_gpu_w4 import acts, dev, rng, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


class Layer:
    def __init__(self, mxq, E, K, I, N, seed):
        mid = 126 - int(round(0.5 * np.log2(K)))  # gate and up values of unit size
        self.E, self.K, self.I, self.N, self.mxq = E, K, I, N, mxq
        self.w13 = weight((E, 2, I), K, seed, lo=mid - 1, hi=mid + 1)
        self.w2 = weight((E, N), I, seed + 1)
        self.p13 = mxq.mxq_prepare_w4(*[t.view(2 * E, I, -1) for t in dev(*self.w13)])
        self.p2 = mxq.mxq_prepare_w4(*dev(*self.w2))

    def values(self):
        f = lambda w: ref.weight_values(w[0].reshape(-1, w[0].shape[-1]), w[1].reshape(-1, w[1].shape[-1]))
        return f(self.w13).reshape(self.E, 2, self.I, self.K), f(self.w2).reshape(self.E, self.N, self.I)

    def __call__(self, a, asf, ids, wt, **kw):
        return self.mxq.mxq_experts_a8w4(*dev(a, asf, ids, wt), self.p13, self.p2, self.I, N=self.N, **kw)


def unit_acts(T, K, seed):
    """Codes of normal rows."""
    from oracle import mx_oracle as O

    return O.group_quant_rows(rng(seed).standard_normal((T, K)).astype(np.float32))


def choose(T, k, E, seed, skew=0.0):
    g = rng(seed)
    like = skew * g.standard_normal(E)
    s = g.standard_normal((T, E)) + like
    ids = np.argsort(-s, axis=1)[:, :k].astype(np.int32)
    return ids, g.random((T, k)).astype(np.float32) * 2 - 0.3


def check(layer, a, asf, ids, wt, out):
    want, tol = ref.experts(ref.act_values(a, asf), ids, wt.astype(np.float64), *layer.values())
    got = out.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


SIZES = [  # T, k, E, K, I, N
    (1, 1, 1, 32, 32, 16), (1, 4, 8, 256, 128, 256), (2, 8, 64, 576, 96, 144), (3, 2, 5, 1024, 160, 1024),
    (7, 3, 4, 4096, 256, 128), (16, 8, 32, 512, 288, 512), (1, 8, 16, 2048, 512, 2048), (33, 2, 3, 384, 128, 272),
    (64, 6, 8, 320, 224, 400), (65, 4, 8, 640, 128, 640), (130, 8, 10, 256, 416, 256), (300, 2, 4, 512, 256, 512),
    (500, 6, 12, 288, 160, 160), (40, 32, 33, 96, 64, 48), (257, 1, 1, 1024, 384, 128), (24, 4, 8, 640, 192, 304),
    (100, 2, 16, 1152, 96, 128), (90, 6, 8, 256, 512, 96), (400, 8, 64, 160, 96, 64), (700, 8, 12, 96, 64, 48),
    (1500, 5, 1000, 64, 32, 32)]


@pytest.mark.parametrize("T,k,E,K,I,N", SIZES)
def test_against_reference(mxq, T, k, E, K, I, N):
    layer = Layer(mxq, E, K, I, N, seed=T + K)
    a, asf = unit_acts(T, K, seed=T + 1)
    ids, wt = choose(T, k, E, seed=T + 2, skew=0.5)
    out = layer(a, asf, ids, wt)
    torch.cuda.synchronize()
    assert mxq.mxq_watchdog_read() == 0
    check(layer, a, asf, ids, wt, out)


@pytest.mark.parametrize("T,k,E,K,I,N", [(1, 8, 128, 512, 256, 512), (1, 16, 16, 4096, 128, 1040), (2, 8, 3, 288, 96, 4096),
                                         (16, 1, 2, 1024, 416, 144), (5, 3, 200, 96, 1024, 80), (3, 5, 1, 640, 32, 272),
                                         (1, 17, 40, 256, 128, 256)])
def test_up_to_sixteen_pairs(mxq, T, k, E, K, I, N):
    """Calls small enough to go without a plan and a sum of their own, and the first that are not."""
    layer = Layer(mxq, E, K, I, N, seed=T + K + E)
    a, asf = unit_acts(T, K, seed=T + 1)
    ids = rng(T + 2).integers(-1, E, (T, k)).astype(np.int32)
    wt = rng(T + 3).random((T, k)).astype(np.float32)
    ws = torch.full((mxq.mxq_experts_workspace_bytes(T, k, E, K, I, N),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # the second finds the first one's arrivals
        out = layer(a, asf, ids, wt, ws=ws)
        check(layer, a, asf, ids, wt, out)
        ids[0] = rng(T + 4).permutation(ids[0])
    out = layer(a, asf, np.full_like(ids, -1), wt, ws=ws)
    assert int(out.count_nonzero()) == 0


@pytest.mark.parametrize("T", [2, 5, 40, 300])
def test_padding_bad_ids_and_repeats(mxq, T):
    E, K, I, N, k = 6, 256, 160, 272, 4
    layer = Layer(mxq, E, K, I, N, seed=1)
    a, asf = unit_acts(T, K, seed=2)
    ids, wt = choose(T, k, E, seed=3)
    ids[T // 2:] = -1                     # padded rows
    ids[0] = 2                            # one expert four times
    ids[1, 2] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = layer(a, asf, ids, wt, err_flag=err)
    assert int(err.item()) == 0
    check(layer, a, asf, ids, wt, out)
    assert int(out[T // 2:].count_nonzero()) == 0
    bad = ids.copy()
    bad[0, 1], bad[1, 0] = E, -2
    out = layer(a, asf, bad, wt, err_flag=err)
    assert int(err.item()) == mxq.MXQ_DEVERR_EXPERT
    check(layer, a, asf, np.where((bad < 0) | (bad >= E), -1, bad), wt, out)


def test_no_row_has_an_expert(mxq):
    layer = Layer(mxq, 4, 128, 64, 144, seed=5)
    a, asf = unit_acts(9, 128, seed=6)
    a[:] = 0x7F  # rows without experts are not read into anything
    out = layer(a, asf, np.full((9, 3), -1, np.int32), np.full((9, 3), np.nan, np.float32))
    assert int(out.count_nonzero()) == 0


@pytest.mark.parametrize("T", [12, 300])
def test_all_rows_on_one_expert(mxq, T):
    layer = Layer(mxq, 7, 288, 128, 128, seed=7)
    a, asf = unit_acts(T, 288, seed=8)
    ids, wt = choose(T, 2, 7, seed=9)
    ids[:] = 5
    check(layer, a, asf, ids, wt, layer(a, asf, ids, wt))


def test_nan_rows_and_stale_workspace(mxq):
    """A NaN row reaches its own output alone, and a workspace full of NaN bytes nothing."""
    for T in (10, 200):
        layer = Layer(mxq, 5, 256, 96, 128, seed=10)
        a, asf = unit_acts(T, 256, seed=11)
        ids, wt = choose(T, 3, 5, seed=12)
        ws = torch.full((mxq.mxq_experts_workspace_bytes(T, 3, 5, 256, 96, 128),), 0xFF, dtype=torch.uint8, device="cuda")
        good = layer(a, asf, ids, wt, ws=ws)
        check(layer, a, asf, ids, wt, good)
        a[4, 100] = 0x7F
        out = layer(a, asf, ids, wt, ws=ws)
        keep = torch.ones(T, dtype=torch.bool)
        keep[4] = False
        assert bool(torch.isnan(out[4]).all()) and torch.equal(out[keep], good[keep])


def test_same_bits_every_time(mxq):
    """The order in which rows are sorted is left to atomics; results are not."""
    layer = Layer(mxq, 8, 512, 256, 512, seed=13)
    for T in (20, 400):
        a, asf = unit_acts(T, 512, seed=14)
        ids, wt = choose(T, 4, 8, seed=15)
        first = layer(a, asf, ids, wt)
        for _ in range(5):
            assert torch.equal(layer(a, asf, ids, wt), first)


def test_side_stream_and_two_graphs_in_turn(mxq):
    """Two captured calls with workspaces of their own, replayed one after the other and at once."""
    layer = Layer(mxq, 8, 288, 128, 288, seed=16)
    T, k = 24, 4
    a, asf = unit_acts(T, 288, seed=17)
    pick = [choose(T, k, 8, seed=18 + i) for i in range(4)]
    want = [layer(a, asf, *p) for p in pick]
    ad, sd = dev(a, asf)
    inp = [dev(*pick[0]), dev(*pick[1])]
    graphs, outs = [], []
    for i in range(2):
        layer.mxq.mxq_experts_a8w4(ad, sd, *inp[i], layer.p13, layer.p2, 128)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.mxq.mxq_experts_a8w4(ad, sd, *inp[i], layer.p13, layer.p2, 128))
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for j in range(4):
        for i in range(2):
            for d, v in zip(inp[i], dev(*pick[(i + j) % 4])):
                d.copy_(v)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[(i + j) % 4])
    s[0].wait_stream(torch.cuda.current_stream())
    got = layer.mxq.mxq_experts_a8w4(ad, sd, *dev(*pick[0]), layer.p13, layer.p2, 128, stream=s[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])


def test_half_of_a_layer(mxq):
    """Norm, router, routing and experts one behind the other, eager and as one graph."""
    T, D, E, k, I = 13, 512, 16, 4, 160
    layer = Layer(mxq, E, D, I, D, seed=30)
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    res = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    w = torch.ones((D,), dtype=torch.bfloat16, device="cuda")
    wr = torch.randint(0, 0x38, (E, D), generator=g, device="cuda", dtype=torch.uint8)
    wr_sf = mxq.mxq_prepare_weight_scales(torch.full((1, E, D // 128), 121, dtype=torch.uint8, device="cuda"), D)
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")

    def step():
        s, y, q, sc = mxq.mxq_add_rms_norm(x, w, residual=res)
        logits = mxq.mxq_linear(y, wr, wr_sf)
        ids, wt = mxq.mxq_route(logits, k, scoring="sigmoid", bias=bias, groups=4, topk_groups=2)
        out = mxq.mxq_experts_a8w4(q, sc, ids, wt, layer.p13, layer.p2, I)
        return s, y, q, sc, logits, ids, wt, out, *mxq.mxq_add_rms_norm(out, w, residual=s)

    s, y, q, sc, logits, ids, wt, out, s2, y2, q2, sc2 = step()
    want, _, _ = ref.route(logits.double().cpu().numpy(), k, "sigmoid", bias=bias.double().cpu().numpy(), groups=4,
                        topk_groups=2)
    assert np.array_equal(ids.cpu().numpy(), want)
    check(layer, q.cpu().numpy(), sc.cpu().numpy(), ids.cpu().numpy(), wt.cpu().numpy(), out)
    assert torch.equal(s2, (out.float() + s.float()).bfloat16())
    eager = [t.clone() for t in (out, s2, y2, q2, sc2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((captured[7], *captured[8:]), eager):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,k,E,K,I,N", [(1, 2, 4, 256, 1024, 128), (1, 1, 3, 128, 4096, 64), (2, 3, 5, 96, 1088, 80),
                                         (1, 3, 6, 64, 2080, 144), (4, 2, 9, 160, 4128, 48), (1, 4, 6, 1024, 1152, 400),
                                         (16, 1, 2, 96, 2048, 272), (8, 2, 5, 128, 1056, 4112)])
def test_few_choices_share_their_columns(mxq, T, k, E, K, I, N):
    """Small calls whose down product gives each choice several parts of I, even and uneven ones."""
    layer = Layer(mxq, E, K, I, N, seed=T + I)
    a, asf = unit_acts(T, K, seed=T + 1)
    ids, wt = choose(T, k, E, seed=T + 2)
    check(layer, a, asf, ids, wt, layer(a, asf, ids, wt))
    ids[0, -1], ids[-1, 0] = -1, E
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = layer(a, asf, ids, wt, err_flag=err)
    assert int(err.item()) == mxq.MXQ_DEVERR_EXPERT and mxq.mxq_watchdog_read() == 0
    check(layer, a, asf, np.where(ids >= E, -1, ids), wt, out)


@pytest.mark.parametrize("T,E,k", [(60, 3, 4), (333, 4, 2), (700, 3, 3), (245, 1, 2)])
def test_tiles_of_one_expert(mxq, T, E, k):
    """Experts of several tiles, of which the last is smaller than the others."""
    layer = Layer(mxq, E, 288, 160, 272, seed=T)
    a, asf = unit_acts(T, 288, seed=T + 1)
    ids = rng(T + 2).integers(0, E, (T, k)).astype(np.int32)
    wt = rng(T + 3).random((T, k)).astype(np.float32)
    check(layer, a, asf, ids, wt, layer(a, asf, ids, wt))
