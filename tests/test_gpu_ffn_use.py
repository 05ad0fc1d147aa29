"""The norm, the routing and the 4-bit products as programs use them: the first call of a process captured into a
graph, calls from two threads at once, and results that lie more than 2^32 elements behind their base."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import ffn_ref as ref
from test_gpu_experts import Layer, check, choose, mxq, unit_acts  # noqa: F401 (mxq: the fixture)
from test_gpu_w4 import dev, weight

pytestmark = pytest.mark.gpu

FIRST = """
import sys
import torch
import mxfp8_block_scaled_inv_gb300 as mxq

name = sys.argv[1]
torch.manual_seed(1)
u = lambda lo, hi, *s: torch.randint(lo, hi, s, device="cuda", dtype=torch.uint8)
x = torch.randn((300, 256), device="cuda").bfloat16()
a, sf = u(0, 0x70, 300, 256), u(118, 124, 300, 2)
blocks = lambda n: u(118, 122, n * 8704)
ids = torch.randint(0, 4, (300, 3), device="cuda", dtype=torch.int32)
wt = torch.rand((300, 3), device="cuda")
w4, w13, w2 = blocks(6), blocks(32), blocks(16)
calls = {
    "norm": lambda: mxq.mxq_add_rms_norm(x, residual=x),
    "route": lambda: mxq.mxq_route(x, 6, scoring="sigmoid", groups=8, topk_groups=4),
    "linear": lambda: (mxq.mxq_linear_a8w4(a, sf, w4, 384),),
    "linear 8": lambda: (mxq.mxq_linear_a8w4(a[:8], sf[:8], w4, 384),),
    "experts": lambda: (mxq.mxq_experts_a8w4(a, sf, ids, wt, w13, w2, 256),),
    "experts 2": lambda: (mxq.mxq_experts_a8w4(a[:2], sf[:2], ids[:2], wt[:2], w13, w2, 256),),
}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = calls[name]()
g.replay()
torch.cuda.synchronize()
want = calls[name]()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, want) if p is not None)
assert mxq.mxq_watchdog_read() == 0
print("as eager")
"""


@pytest.mark.parametrize("name", ["norm", "route", "linear", "linear 8", "experts", "experts 2"])
def test_the_first_call_of_a_process_is_captured(mxq, name):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST, name], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as eager" in r.stdout, r.stderr[-2000:]


def test_two_threads_at_once(mxq):
    layer = Layer(mxq, 8, 512, 256, 512, seed=40)
    inputs = [(*unit_acts(T, 512, seed=T), *choose(T, 4, 8, seed=T + 1)) for T in (3, 700)]
    want = [layer(*i) for i in inputs]
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                args = dev(*inputs[i])
                for _ in range(50):
                    got = mxq.mxq_experts_a8w4(*args, layer.p13, layer.p2, layer.I)
                    y = mxq.mxq_add_rms_norm(got)[1]
                    if not torch.equal(got, want[i]) or y.shape != got.shape:
                        failed.append(i)
        except Exception as e:  # reported by the main thread
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def room(need):
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs more memory")


def test_linear_past_32_bits(mxq):
    T, N, K = 264000, 16384, 96
    room(30 << 30)
    w = weight((N,), K, seed=50)
    w4 = mxq.mxq_prepare_w4(*dev(*w))
    a, asf = unit_acts(512, K, seed=51)
    pick = np.random.Generator(np.random.PCG64(52)).integers(0, 512, T)
    at = torch.from_numpy(pick).cuda()
    ad, sd = dev(a, asf)
    out = mxq.mxq_linear_a8w4(ad[at], sd[at], w4, N)
    want, mag = ref.linear(ref.act_values(a, asf), ref.weight_values(*w))
    for t in (0, 1, 131071, 131072, 262143, 262144, T - 241, T - 1):
        v = want[pick[t]]
        tol = 1e-5 * mag[pick[t]] + 2.0 ** -8 * np.abs(v) + 2.0 ** -126
        assert np.all(np.abs(out[t].double().cpu().numpy() - v) <= tol), t
    # Equal rows have equal results wherever they lie.
    first = torch.empty(512, dtype=torch.long, device="cuda").scatter_(0, at.flip(0), torch.arange(T - 1, -1, -1, device="cuda"))
    for t0 in range(0, T, 33000):
        assert torch.equal(out[t0:t0 + 33000], out[first[at[t0:t0 + 33000]]])


def test_experts_past_32_bits(mxq):
    T, k, E, K, I, N = 140000, 4, 6, 96, 64, 8192
    room(40 << 30)
    layer = Layer(mxq, E, K, I, N, seed=60)
    a, asf = unit_acts(300, K, seed=61)
    ids, wt = choose(300, k, E, seed=62)
    at = torch.from_numpy(np.random.Generator(np.random.PCG64(63)).integers(0, 300, T)).cuda()
    at[:300] = torch.arange(300, device="cuda")
    ad, sd, idd, wd = dev(a, asf, ids, wt)
    out = mxq.mxq_experts_a8w4(ad[at], sd[at], idd[at], wd[at], layer.p13, layer.p2, I, N=N)
    check(layer, a, asf, ids, wt, out[:300])
    for t0 in range(0, T, 20000):
        assert torch.equal(out[t0:t0 + 20000], out[at[t0:t0 + 20000]])


def test_between_kernels_that_begin_early(mxq):
    """4-bit products between a long kernel and others that begin beside them: the same results as one by one."""
    g = torch.Generator(device="cuda")
    g.manual_seed(70)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    long, w4 = r(16384, 4096), mxq.mxq_prepare_w4(*dev(*weight((4096,), 4096, seed=71)))
    layer = Layer(mxq, 8, 4096, 1024, 4096, seed=72)
    ids, wt = dev(*choose(1, 2, 8, seed=73))
    q, cache = r(8, 16, 128), r(4096, 128)
    table = torch.arange(64, device="cuda", dtype=torch.int32).view(8, 8)
    lens = torch.full((8,), 500, device="cuda", dtype=torch.int32)
    w8 = torch.randint(0, 0x38, (256, 4096), generator=g, device="cuda", dtype=torch.uint8)
    w8_sf = mxq.mxq_prepare_weight_scales(torch.full((1, 256, 32), 121, dtype=torch.uint8, device="cuda"), 4096)

    def steps(sync):
        _, y, codes, sf = mxq.mxq_add_rms_norm(long)
        sync()
        out = [y[:3]]
        for _ in range(3):
            out.append(mxq.mxq_linear_a8w4(codes[:1], sf[:1], w4, 4096))
            sync()
            out.append(mxq.mxq_attn(q, cache, table, lens))
            sync()
            out.append(mxq.mxq_experts_a8w4(codes[:1], sf[:1], ids, wt, layer.p13, layer.p2, 1024))
            sync()
            out.append(mxq.mxq_linear(y[:2], w8, w8_sf))
            sync()
        return out

    want = steps(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = steps(lambda: None)
    for _ in range(3):
        got = steps(lambda: None)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, captured):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert mxq.mxq_watchdog_read() == 0
