"""What a call of the binding allocates belongs to the stream that it runs on:
memory taken from another stream's pool may still be in use there, and may be
handed out again there while the call's kernels use it.  Checked on the CPU,
with the library's entry points and the streams replaced by recorders."""

import contextlib
import types

import pytest
import torch

import mxfp8_block_scaled_inv_gb300 as mxq

WS = 4096


class Recorder:
    """Stands in for torch in the binding: tensors on the CPU, with the stream current at their allocation."""

    def __init__(self):
        self.now, self.allocs = "current", []
        self.cuda = types.SimpleNamespace(stream=self.stream, current_stream=lambda *a: side("current"))

    def __getattr__(self, name):
        return getattr(torch, name)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s.name
        yield
        self.now = before

    def empty(self, *a, **kw):
        self.allocs.append(self.now)
        return torch.empty(*a, **{**kw, "device": "cpu"})

    def empty_like(self, t):
        self.allocs.append(self.now)
        return torch.empty_like(t)


def side(name):
    return types.SimpleNamespace(name=name, cuda_stream=7)


class Library:
    """Entry points that succeed; sizes that call for a workspace."""

    def __getattr__(self, name):
        return (lambda *a: WS) if name.endswith("_bytes") else (lambda *a: 0)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(mxq, "torch", r)
    monkeypatch.setattr(mxq, "lib", lambda: Library())
    monkeypatch.setattr(mxq, "_tensor", lambda fn, name, t, *a: 0)
    monkeypatch.setattr(mxq, "_raw_stream", None)
    return r


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


CALLS = {
    "inv_rope_group_quant": (lambda **k: mxq.mxq_inv_rope_group_quant(bf(4, 2, 128), **k), 2),
    "prepare_weight_scales": (lambda **k: mxq.mxq_prepare_weight_scales(u8(2, 128, 1), 128, **k), 1),
    "bmm_a8w8": (lambda **k: mxq.mxq_bmm_a8w8(u8(4, 2, 128), u8(4, 2, 1), u8(2, 128, 128), u8(WS), **k), 2),
    "linear": (lambda **k: mxq.mxq_linear(bf(4, 128), u8(128, 128), u8(WS), **k), 2),
    "linear_noalloc": (lambda **k: mxq.mxq_linear_noalloc(bf(4, 128), u8(128, 128), u8(WS), **k), 1),
    "dequant_bf16": (lambda **k: mxq.mxq_dequant_bf16(u8(2, 128, 128), u8(2, 128, 1), **k), 1),
    "scales_f32_to_e8m0": (lambda **k: mxq.mxq_scales_f32_to_e8m0(torch.ones(4), **k), 1),
    "wo_a": (lambda **k: mxq.mxq_wo_a(bf(4, 2, 128), None, None, None, u8(2, 128, 128), u8(WS), R=0, **k), 2),
    "rope_kv_insert": (lambda **k: mxq.mxq_rope_kv_insert(bf(4, 2, 64), bf(4, 64), None, None, None, 0,
                                                          torch.zeros(4, dtype=torch.int64), bf(8, 64), **k), 1),
    "rope_kv4_insert": (lambda **k: mxq.mxq_rope_kv4_insert(bf(4, 2, 64), bf(4, 64), None, None, None, 0,
                                                            torch.zeros(4, dtype=torch.int64), u8(8, 32), u8(8, 2),
                                                            **k), 1),
    "kv4_gather": (lambda **k: mxq.mxq_kv4_gather(u8(8, 32), u8(8, 2), torch.zeros(4, dtype=torch.int64), **k), 1),
    "attn": (lambda **k: mxq.mxq_attn(bf(4, 2, 64), bf(64, 64), torch.zeros((4, 1), dtype=torch.int32),
                                      torch.zeros(4, dtype=torch.int32), **k), 2),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_given_stream(rec, name):
    call, n = CALLS[name]
    call(stream=side("side"))
    assert rec.allocs == ["side"] * n and rec.now == "current"


@pytest.mark.parametrize("name", CALLS)
def test_allocations_without_a_stream(rec, name):
    call, n = CALLS[name]
    call()
    assert rec.allocs == ["current"] * n
