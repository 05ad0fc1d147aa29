"""Refusals of mxq_add_rms_norm, mxq_route, mxq_prepare_w4, mxq_linear_a8w4 and mxq_experts_a8w4 without a GPU:
each invalid argument returns its documented status and launches nothing."""

import ctypes

import pytest
import torch


def at(a):
    return ctypes.c_void_p(a) if a else None


X, R, S, W, Y, Q, C = (i << 36 for i in range(1, 8))  # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from mxfp8_block_scaled_inv_gb300 import build as B

    B.build()
    import mxfp8_block_scaled_inv_gb300 as mxq

    return mxq.lib()


NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


def norm(L, x=X, r=R, s=S, w=W, T=8, D=4096, eps=1e-6, y=Y, q=Q, c=C):
    return L.mxq_add_rms_norm(at(x), at(r), at(s), at(w), T, D, eps, at(y), at(q), at(c), None)


def test_norm_argument_errors(L):
    for bad in (dict(x=None), dict(r=None), dict(s=None), dict(q=None), dict(c=None), dict(y=None, q=None, c=None)):
        assert norm(L, **bad) == 1, bad
    for bad in (dict(T=-1), dict(D=0), dict(D=8), dict(D=4100), dict(eps=0.0), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(L, **bad) == 2, bad
    for bad in (dict(D=65552), dict(T=1 << 31)):
        assert norm(L, **bad) == 4, bad
    for name, v in (("x", X), ("r", R), ("s", S), ("w", W), ("y", Y), ("q", Q)):
        assert norm(L, **{name: v + 8}) == 3, name
    assert norm(L, T=0, x=None, r=None, s=None, y=None, q=None, c=None) == 0


def test_norm_overlaps(L):
    n = 8 * 4096 * 2
    for bad in (dict(s=X + 16), dict(s=R - 16), dict(y=X + n - 16), dict(y=S), dict(y=S + n - 16), dict(q=X),
                dict(q=Y + 16), dict(c=Q), dict(s=W), dict(y=W + 16), dict(q=W), dict(s=R, y=R), dict(c=X + n - 1)):
        assert norm(L, **bad) == 2, bad


@NO_GPU
def test_norm_accepted(L):
    n = 8 * 4096 * 2
    for good in (dict(), dict(s=R), dict(s=X), dict(y=X), dict(y=R), dict(s=R, y=X), dict(s=X, y=R), dict(w=None),
                 dict(y=None), dict(q=None, c=None), dict(r=None, s=None), dict(r=None, s=None, y=X), dict(s=X + n),
                 dict(c=C + 1), dict(D=16), dict(D=65536)):
        assert norm(L, **good) == 7, good


def route(L, l=X, dt=0, T=4, E=256, b=R, k=8, sc=1, G=8, keep=4, top=2, ren=1, scale=1.0, ids=S, w=W):
    return L.mxq_route(at(l), dt, T, E, at(b), k, sc, G, keep, top, ren, scale, at(ids), at(w), None)


def test_route_argument_errors(L):
    for name in ("l", "ids", "w"):
        assert route(L, **{name: None}) == 1, name
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=257), dict(G=0), dict(G=7), dict(keep=0), dict(keep=9),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=X), dict(w=X + 16), dict(w=S),
                dict(ids=R), dict(w=R + 1020), dict(ids=X + 4 * 256 * 4 - 4)):
        assert route(L, **bad) == 2, bad
    for bad in (dict(E=2048), dict(k=33), dict(E=512, G=64), dict(dt=2), dict(sc=3), dict(sc=-1), dict(top=0),
                dict(top=3), dict(T=1 << 31)):
        assert route(L, **bad) == 4, bad
    for bad in (dict(l=X + 8), dict(b=R + 2), dict(ids=S + 2), dict(w=W + 1)):
        assert route(L, **bad) == 3, bad
    assert route(L, T=0, l=None, ids=None, w=None) == 0


@NO_GPU
def test_route_accepted(L):
    for good in (dict(), dict(b=None), dict(dt=1), dict(sc=0), dict(sc=2), dict(G=1, keep=1), dict(E=1, k=1, G=1, keep=1),
                 dict(E=1024, G=32, k=32), dict(E=60, G=5, keep=5, k=6), dict(ids=S + 4)):
        assert route(L, **good) == 7, good


def prepare(L, w=X, s=R, B=2, N=200, K=576, out=S):
    return L.mxq_prepare_w4(at(w), at(s), B, N, K, at(out), None)


def test_w4_bytes(L):
    assert L.mxq_w4_bytes(1, 1, 32) == 8704 and L.mxq_w4_bytes(3, 129, 160) == 3 * 2 * 2 * 8704
    assert L.mxq_w4_bytes(1, 128, 65536) == 512 * 8704
    for bad in ((0, 128, 128), (1, 0, 128), (1, 128, 0), (1, 128, 48), (1, 128, 65568), (1 << 30, 1 << 30, 65536),
                ((1 << 31) // 136 + 1, 128, 128), (-1, 128, 128), (1, -5, 128)):
        assert L.mxq_w4_bytes(*bad) == 0, bad


def test_prepare_argument_errors(L):
    for name in ("w", "s", "out"):
        assert prepare(L, **{name: None}) == 1, name
    for bad in (dict(B=0), dict(N=0), dict(K=16), dict(K=600), dict(out=X), dict(out=R), dict(out=X + 2 * 200 * 288 - 32)):
        assert prepare(L, **bad) == 2, bad
    for bad in (dict(K=65568), dict(B=1 << 30, N=1 << 30)):
        assert prepare(L, **bad) == 4, bad
    for bad in (dict(w=X + 8), dict(out=S + 16)):
        assert prepare(L, **bad) == 3, bad


def linear(L, a=X, s=R, w=W, out=Y, T=4, N=5120, K=576):
    return L.mxq_linear_a8w4(at(a), at(s), at(w), at(out), T, N, K, None)


def test_linear_argument_errors(L):
    for name in ("a", "s", "w", "out"):
        assert linear(L, **{name: None}) == 1, name
    for bad in (dict(T=-1), dict(N=0), dict(N=24), dict(K=0), dict(K=48), dict(out=X), dict(out=X + 4 * 576 - 16),
                dict(out=R), dict(out=W), dict(out=W + 5120 // 128 * 5 * 8704 - 32)):
        assert linear(L, **bad) == 2, bad
    for bad in (dict(K=65568), dict(T=1 << 31), dict(N=1 << 30, K=576), dict(T=(1 << 31) - 1, N=1 << 20)):
        assert linear(L, **bad) == 4, bad
    for bad in (dict(a=X + 8), dict(out=Y + 8), dict(w=W + 16)):
        assert linear(L, **bad) == 3, bad
    assert linear(L, T=0, a=None, out=None) == 0


def experts(L, a=X, s=R, ids=S, wt=W, w13=Y, w2=Q, out=C, T=4, k=8, E=16, K=576, I=288, N=1024, err=None, ws=8 << 36,
            nbytes=1 << 34):
    return L.mxq_experts_a8w4(at(a), at(s), at(ids), at(wt), at(w13), at(w2), at(out), T, k, E, K, I, N, at(err), at(ws),
                              nbytes, None)


def test_experts_argument_errors(L):
    for name in ("a", "s", "ids", "wt", "w13", "w2", "out"):
        assert experts(L, **{name: None}) == 1, name
    need = L.mxq_experts_workspace_bytes(4, 8, 16, 576, 288, 1024)
    assert need > 0
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(K=0), dict(K=48), dict(I=0), dict(I=48), dict(N=0), dict(N=24),
                dict(out=X), dict(out=S), dict(out=Y), dict(out=8 << 36), dict(ws=X), dict(ws=C), dict(ws=Q),
                dict(ws=W - need + 16)):
        assert experts(L, **bad) == 2, bad
    for bad in (dict(k=33), dict(E=1025), dict(K=65568), dict(I=65568), dict(T=1 << 21), dict(T=1 << 40),
                dict(E=1024, N=1 << 30, I=65536), dict(E=1024, I=65536, K=65536)):
        assert experts(L, **bad) == 4, bad
    for bad in (dict(ws=None), dict(nbytes=need - 1)):
        assert experts(L, **bad) == 6, bad
    for bad in (dict(a=X + 8), dict(out=C + 8), dict(w13=Y + 16), dict(w2=Q + 16), dict(ids=S + 2), dict(wt=W + 2),
                dict(err=(1 << 20) + 2), dict(ws=(8 << 36) + 8)):
        assert experts(L, **bad) == 3, bad
    assert experts(L, T=0, a=None, out=None, ws=None) == 0


def test_error_words_in_other_buffers_and_weights_past_the_coordinates(L):
    """An error word in the workspace or the output; 2^24 blocks of a tall and narrow weight."""
    for err in (8 << 36, (8 << 36) + 512, C, C + 2 * 4 * 1024 - 4):
        assert experts(L, err=err) == 2, err
    assert linear(L, N=(1 << 31) - 16, K=32, T=1) == 4 and prepare(L, B=1, N=(1 << 31) - 16, K=32) == 4


def test_experts_workspace(L):
    f = L.mxq_experts_workspace_bytes
    good = (4, 8, 16, 576, 288, 1024)
    for at, v in ((0, -1), (1, 0), (1, 33), (2, 0), (2, 1025), (3, 48), (3, 0), (4, 48), (5, 24), (0, 1 << 21)):
        bad = good[:at] + (v,) + good[at + 1:]
        assert f(*bad) == 0, bad
    assert f(8, *good[1:]) > f(*good)


@NO_GPU
def test_valid_calls_without_device(L):
    assert prepare(L) == 7 and linear(L) == 7 and experts(L) == 7
    assert linear(L, T=8192, N=16, K=32) == 7 and linear(L, s=R + 1) == 7
    assert experts(L, s=R + 1, err=1 << 20, nbytes=L.mxq_experts_workspace_bytes(4, 8, 16, 576, 288, 1024)) == 7
    assert experts(L, k=1, E=1, K=32, I=32, N=16) == 7
