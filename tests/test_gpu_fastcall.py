"""The binding's quick way in (mxq_fastcall) gives what its Python code gives: the same outputs, on the current
stream, in a captured graph, and the same refusals."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


def inputs(mxq, T=5):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)
    x, res, w = r(T, 256).bfloat16(), r(T, 256).bfloat16(), r(256).bfloat16()
    logits, bias = r(T, 8), r(8)
    a, sf = u(0, 0x70, T, 256), u(118, 124, T, 2)
    w4 = mxq.mxq_prepare_w4(u(0, 255, 144, 128), u(118, 122, 144, 8))
    w13 = mxq.mxq_prepare_w4(u(0, 255, 16, 96, 128), u(112, 114, 16, 96, 8))
    w2 = mxq.mxq_prepare_w4(u(0, 255, 8, 256, 48), u(118, 122, 8, 256, 3))
    ids, wt = mxq.mxq_route(logits, 2)
    return {
        "norm": lambda: mxq.mxq_add_rms_norm(x, w, 1e-5, residual=res),
        "norm codes": lambda: mxq.mxq_add_rms_norm(x, None, 1, want_y=False),
        "norm y": lambda: mxq.mxq_add_rms_norm(x.view(T, 2, 128), w[:128], want_codes=False),
        "route": lambda: mxq.mxq_route(logits, 3, scoring="sigmoid", bias=bias, groups=4, topk_groups=2, scale=2),
        "route bf16": lambda: mxq.mxq_route(logits.bfloat16(), 3, renormalise=0),
        "linear": lambda: mxq.mxq_linear_a8w4(a, sf, w4, 144),
        "experts": lambda: mxq.mxq_experts_a8w4(a, sf, ids, wt, w13, w2, 96),
        "experts N": lambda: mxq.mxq_experts_a8w4(a, sf, ids, wt, w13, w2, 96, 256),
    }


def same(a, b):
    a, b = (a, b) if isinstance(a, tuple) else ((a,), (b,))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


@pytest.mark.parametrize("T", [0, 1, 5, 40])
def test_same_results(mxq, monkeypatch, T):
    assert mxq._fastcall()
    calls = inputs(mxq, T)
    quick = {n: f() for n, f in calls.items()}
    monkeypatch.setattr(mxq, "_fast", False)
    monkeypatch.setattr(mxq, "_fastcall", lambda: False)
    for n, f in calls.items():
        same(quick[n], f())


def test_current_stream_and_graph(mxq):
    calls = inputs(mxq)
    want = {n: f() for n, f in calls.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = {n: f() for n, f in calls.items()}
    side.synchronize()
    for n in calls:
        same(got[n], want[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = {n: f() for n, f in calls.items()}
    graph.replay()
    torch.cuda.synchronize()
    for n in calls:
        same(got[n], want[n])


def test_parameters_and_refusals(mxq):
    x = torch.randn((4, 256), device="cuda").bfloat16()
    w = torch.nn.Parameter(torch.ones(256, device="cuda", dtype=torch.bfloat16), requires_grad=False)
    same(mxq.mxq_add_rms_norm(x, w), mxq.mxq_add_rms_norm(x, None))
    for bad in (lambda: mxq.mxq_add_rms_norm(x.t()), lambda: mxq.mxq_add_rms_norm(x[:, :100]),
                lambda: mxq.mxq_add_rms_norm(x.float()), lambda: mxq.mxq_add_rms_norm(x, eps=0.0),
                lambda: mxq.mxq_add_rms_norm(x, want_y=False, want_codes=False),
                lambda: mxq.mxq_add_rms_norm(x, x), lambda: mxq.mxq_add_rms_norm(x, residual=x[:2]),
                lambda: mxq.mxq_add_rms_norm(x[:, :24].contiguous()), lambda: mxq.mxq_route(x, 0),
                lambda: mxq.mxq_route(x, 257), lambda: mxq.mxq_route(x, 2, scoring="none"),
                lambda: mxq.mxq_route(x, 2, groups=3), lambda: mxq.mxq_route(x, 2, bias=x[0]),
                lambda: mxq.mxq_route(x[0], 2)):
        with pytest.raises((mxq.MxqError, ValueError)):
            bad()
