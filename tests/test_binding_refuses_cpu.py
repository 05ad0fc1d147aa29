"""What the binding of the attention and 4-bit cache functions refuses before the library is called: an
address that the kernels would write to, or read from, in the wrong memory or with the wrong width."""

import types

import pytest
import torch

import mxfp8_block_scaled_inv_gb300 as mxq
from mxfp8_block_scaled_inv_gb300 import build


class Dev:
    """Looks like a contiguous CUDA tensor to the binding."""

    def __init__(self, shape, dtype, cuda=True, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self._c = torch.Size(shape), dtype, cuda, contiguous
        self.device = types.SimpleNamespace(index=0)

    def is_contiguous(self):
        return self._c

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if i is None else s[i]

    def data_ptr(self):
        return 1 << 20


class Library:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("mxq_status_string", "mxq_last_error"):
            return getattr(self.real, name)

        def call(*a):
            self.calls.append((name, a))
            if name.endswith("_bytes"):
                return 4096
            return 1 if "insert" in name and a[12] > 0 and None in a[7:10] else 0  # pos, cos or sin with R > 0

        return call


@pytest.fixture
def lib(monkeypatch):
    build.build()
    fake = Library(mxq.lib())
    monkeypatch.setattr(mxq, "lib", lambda: fake)
    monkeypatch.setattr(mxq, "_stream_of", lambda *a: 0)
    return fake


B16, U8, I32, I64, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


def attn(**kw):
    a = dict(q=Dev((4, 2, 64), B16), cache=Dev((64, 64), U8), block_table=Dev((4, 1), I32), seq_lens=Dev((4,), I32),
             kv_scale=Dev((1,), F32), out=Dev((4, 2, 64), B16), ws=Dev((4096,), U8), err_flag=Dev((1,), I32))
    return mxq.mxq_attn(**{**a, **kw})


def insert(**kw):
    a = dict(q=Dev((4, 2, 64), B16), kv=Dev((4, 64), B16), pos=Dev((4,), I64), cos=Dev((9, 32), B16),
             sin=Dev((9, 32), B16), R=64, slot_mapping=Dev((4,), I64), cache=Dev((8, 32), U8), cache_sf=Dev((8, 2), U8),
             q_out=Dev((4, 2, 64), B16), err_flag=Dev((1,), I32))
    return mxq.mxq_rope_kv4_insert(**{**a, **kw})


def gather(**kw):
    a = dict(cache=Dev((8, 32), U8), cache_sf=Dev((8, 2), U8), slots=Dev((4,), I64), out=Dev((4, 64), B16),
             err_flag=Dev((1,), I32))
    return mxq.mxq_kv4_gather(**{**a, **kw})


@pytest.mark.parametrize("call", [attn, insert, gather])
def test_good_calls_reach_the_library(lib, call):
    call()
    call(err_flag=None)
    assert len(lib.calls) == 2


@pytest.mark.parametrize("call", [attn, insert, gather])
@pytest.mark.parametrize("flag", [Dev((1,), I32, cuda=False), Dev((1,), I64), Dev((0,), I32), Dev((1,), F32)])
def test_err_flag(lib, call, flag):
    with pytest.raises(mxq.MxqError):
        call(err_flag=flag)
    assert not lib.calls


@pytest.mark.parametrize("ws", [Dev((4096,), U8, cuda=False), Dev((4096,), U8, contiguous=False), Dev((4096,), F32)])
def test_workspace(lib, ws):
    with pytest.raises(mxq.MxqError):
        attn(ws=ws)
    assert not lib.calls


@pytest.mark.parametrize("scale", [Dev((1,), F32, cuda=False), Dev((0,), F32), Dev((1,), B16)])
def test_kv_scale(lib, scale):
    with pytest.raises(mxq.MxqError):
        attn(kv_scale=scale)
    assert not lib.calls


@pytest.mark.parametrize("name", ["pos", "cos", "sin"])
def test_missing_rotation_tables(lib, name):
    """The library answers, with an MxqError like any other."""
    with pytest.raises(mxq.MxqError):
        insert(**{name: None})
    insert(pos=None, cos=None, sin=None, R=0)
