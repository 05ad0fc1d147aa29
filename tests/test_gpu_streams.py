"""Calls on a stream of their own through the `stream` argument: what they allocate is not handed out to
the current stream while their kernels are still to run."""

import pytest
import torch

from test_gpu_attn import Problem, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
def test_attn_on_given_streams(mxq, cache):
    """Two side streams that are held up by some milliseconds, each with a call whose keys are split (a
    workspace of partial sums); meanwhile the current stream fills tensors of the workspace's and the
    output's size."""
    p = Problem([1, 1], [3000, 2000], 16, 512, cache, seed=3000)
    want = p.want()
    d = "cuda"
    q, kv, bt = p.q.to(d), p.kv.to(d), torch.from_numpy(p.bt).to(d)
    lens = torch.tensor(p.lens, dtype=torch.int32, device=d)
    kw = dict(page_size=p.page, kv_scale=torch.tensor([0.0371], device=d) if cache == "e4m3" else None,
              cache_sf=None if p.sf is None else p.sf.to(d))
    need = mxq.mxq_attn_workspace_bytes(2, 2, 16, 512, p.pages, p.page)
    assert need > 0
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(10_000_000)
        outs.append(mxq.mxq_attn(q, kv, bt, lens, stream=s, **kw))
    filled = [torch.full((n,), 0xFF, dtype=torch.uint8, device=d) for n in 4 * [need, 2 * q.numel()]]
    torch.cuda.synchronize()
    for out in outs:
        check(out, None, want)
    assert all(bool((f == 0xFF).all()) for f in filled)
    assert mxq.mxq_watchdog_read() == 0


def test_wo_a_on_a_given_stream(mxq):
    """The projection's codes and scales (a workspace from 33 tokens on) likewise; the same bits as on the
    current stream."""
    T, G, D, N, d = 96, 2, 256, 128, "cuda"
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, G, D), generator=g).bfloat16().to(d)
    w = torch.randn((G, N, D), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(d)
    w_sf = mxq.mxq_prepare_weight_scales(torch.full((G, N, 2), 127, dtype=torch.uint8, device=d), D)
    want = mxq.mxq_wo_a(x, None, None, None, w, w_sf, R=0)
    need = mxq.mxq_wo_a_workspace_bytes(T, G, D, N)
    assert need > 0
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(10_000_000)
    out = mxq.mxq_wo_a(x, None, None, None, w, w_sf, R=0, stream=s)
    filled = [torch.full((n,), 0xFF, dtype=torch.uint8, device=d) for n in 4 * [need, 2 * T * G * N]]
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert all(bool((f == 0xFF).all()) for f in filled)
