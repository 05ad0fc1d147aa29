"""Refusals of mxq_attn, mxq_rope_kv4_insert and mxq_kv4_gather without a GPU:
each invalid argument returns its documented status and launches nothing."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p(1 << 20)        # 16-byte aligned, never dereferenced
Q = ctypes.c_void_p(1 << 30)
U = ctypes.c_void_p((1 << 20) + 8)  # 8-byte aligned only
V = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    from mxfp8_block_scaled_inv_gb300 import build as B

    B.build()
    import mxfp8_block_scaled_inv_gb300 as mxq

    return mxq.lib()


def attn(L, q=P, T=4, H=64, D=512, q_start=P, seq_lens=P, B=4, bt=P, max_pages=8, page=64, kv=P, slots=4096,
         dtype=1, scale=P, sf=P, window=0, sinks=0, sm=0.1, out=Q, lse=None, err=None, ws=P, ws_bytes=1 << 40):
    return L.mxq_attn(q, T, H, D, q_start, seq_lens, B, bt, max_pages, page, kv, slots, dtype, scale, sf, window,
                      sinks, sm, out, lse, err, ws, ws_bytes, None)


def test_attn_argument_errors(L):
    for name in ("q", "seq_lens", "bt", "kv", "out"):
        assert attn(L, **{name: None}) == 1, name
    assert attn(L, dtype=0, scale=None) == 1
    assert attn(L, dtype=2, sf=None) == 1
    for bad in (dict(T=-1), dict(H=0), dict(B=0), dict(D=32), dict(max_pages=0), dict(page=0), dict(page=24),
                dict(page=8), dict(window=-1), dict(sinks=-1), dict(slots=0), dict(sm=float("inf")),
                dict(sm=float("nan")), dict(q_start=None, T=3)):
        assert attn(L, **bad) == 2, bad
    for bad in (dict(D=576), dict(D=96), dict(H=4097), dict(dtype=3), dict(dtype=-1), dict(T=1 << 31),
                dict(T=1 << 25, H=64), dict(T=1 << 62, H=4096), dict(max_pages=1 << 25, page=64),
                dict(slots=1 << 40)):
        assert attn(L, **bad) == 4, bad
    for bad in (dict(q=U), dict(kv=U), dict(out=U), dict(q_start=V), dict(seq_lens=V), dict(bt=V), dict(scale=V),
                dict(lse=V), dict(err=V)):
        assert attn(L, **bad) == 3, bad
    assert attn(L, T=0, q=None, kv=None, out=None) == 0


def test_attn_workspace(L):
    need = L.mxq_attn_workspace_bytes(1, 1, 64, 512, 2048, 64, 0, 0)  # 131,072 keys of one row tile: split
    args = dict(T=1, B=1, max_pages=2048)
    if need:
        assert attn(L, **args, ws=None) == 6
        assert attn(L, **args, ws_bytes=need - 1) == 6
        assert attn(L, **args, ws=U, ws_bytes=need) == 3
    # Sizes that mxq_attn refuses need none.
    assert L.mxq_attn_workspace_bytes(1, 1, 64, 500, 2048, 64, 0, 0) == 0
    assert L.mxq_attn_workspace_bytes(-1, 1, 64, 512, 2048, 64, 0, 0) == 0
    # Never less for more keys or more tokens at the same batch.
    assert L.mxq_attn_workspace_bytes(1, 1, 64, 512, 1, 64, 0, 0) <= need


def kv4(L, q=P, q_out=Q, T=4, H=2, Dq=512, kv=P, Dk=512, pos=P, cos=P, sin=P, cs_ld=32, max_pos=16, R=64, slot=P,
        cache=P, sf=P, num_slots=8, err=None):
    return L.mxq_rope_kv4_insert(q, q_out, T, H, Dq, kv, Dk, pos, cos, sin, cs_ld, max_pos, R, slot, cache, sf,
                                 num_slots, err, None)


def test_kv4_insert_argument_errors(L):
    for name in ("kv", "slot", "cache", "sf", "q", "q_out", "pos", "cos", "sin"):
        assert kv4(L, **{name: None}) == 1, name
    for bad in (dict(Dk=16), dict(Dk=528), dict(Dq=520), dict(T=-1), dict(num_slots=-1), dict(cs_ld=16),
                dict(max_pos=0), dict(q_out=ctypes.c_void_p((1 << 20) + 1024))):
        assert kv4(L, **bad) == 2, bad
    for bad in (dict(R=8), dict(R=528), dict(Dq=256, R=272), dict(T=1 << 31), dict(T=1 << 20, H=64)):
        assert kv4(L, **bad) == 4, bad
    for bad in (dict(kv=U), dict(q=U), dict(q_out=U), dict(cache=U), dict(cs_ld=36), dict(slot=V), dict(err=V)):
        assert kv4(L, **bad) == 3, bad
    assert kv4(L, T=0, kv=None, cache=None) == 0


def gather(L, cache=P, sf=P, num_slots=8, Dk=64, slots=P, n=4, out=Q, err=None):
    return L.mxq_kv4_gather(cache, sf, num_slots, Dk, slots, n, out, err, None)


def test_kv4_gather_argument_errors(L):
    for name in ("cache", "sf", "slots", "out"):
        assert gather(L, **{name: None}) == 1, name
    for bad in (dict(n=-1), dict(num_slots=-1), dict(Dk=16), dict(Dk=48)):
        assert gather(L, **bad) == 2, bad
    assert gather(L, n=1 << 31) == 4 and gather(L, n=1 << 28, Dk=64) == 4
    for bad in (dict(cache=U), dict(out=U), dict(slots=V), dict(err=V)):
        assert gather(L, **bad) == 3, bad
    assert gather(L, n=0, cache=None) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_device(L):
    assert attn(L) == 7 and attn(L, dtype=0) == 7 and attn(L, dtype=2, q_start=None) == 7
    assert kv4(L) == 7 and kv4(L, q=None, q_out=None, H=0, Dq=0) == 7 and gather(L) == 7
