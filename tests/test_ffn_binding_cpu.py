"""What the binding of the norm, routing and 4-bit functions refuses before the library is called, whose memory it
allocates from, and that its quick way in leaves everything but the common case to the Python code."""

import contextlib
import types

import pytest
import torch

import mxfp8_block_scaled_inv_gb300 as mxq
from mxfp8_block_scaled_inv_gb300 import build

B16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class Dev:
    """Looks like a contiguous CUDA tensor to the binding."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self.dev, self._c = torch.Size(shape), dtype, device, contiguous
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self._c

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


class Library:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("mxq_status_string", "mxq_last_error") or name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*a):
            self.calls.append((name, a))
            return 0

        return call


@pytest.fixture
def lib(monkeypatch):
    build.build()
    fake = Library(mxq.lib())
    monkeypatch.setattr(mxq, "lib", lambda: fake)
    monkeypatch.setattr(mxq, "_fast", False)
    monkeypatch.setattr(mxq, "_fastcall", lambda: False)
    monkeypatch.setattr(mxq, "_stream_on", lambda *a: 0)
    monkeypatch.setattr(mxq, "_current_device", lambda: 0)
    return fake


def norm(**kw):
    a = dict(x=Dev((4, 256), B16), weight=Dev((256,), B16), residual=Dev((4, 256), B16),
             residual_out=Dev((4, 256), B16), y=Dev((4, 256), B16), q=Dev((4, 256), U8), sc=Dev((4, 2), U8))
    return mxq.mxq_add_rms_norm(**{**a, **kw})


def route(**kw):
    a = dict(logits=Dev((4, 64), F32), k=6, bias=Dev((64,), F32), ids=Dev((4, 6), I32), weights=Dev((4, 6), F32))
    return mxq.mxq_route(**{**a, **kw})


def prepare(**kw):
    a = dict(w=Dev((2, 128, 64), U8), w_e8m0=Dev((2, 128, 4), U8), out=Dev((2 * 8704,), U8))
    return mxq.mxq_prepare_w4(**{**a, **kw})


def linear(**kw):
    a = dict(a=Dev((4, 288), U8), a_sf=Dev((4, 3), U8), w4=Dev((3 * 8704,), U8), N=128, out=Dev((4, 128), B16))
    return mxq.mxq_linear_a8w4(**{**a, **kw})


def experts(**kw):
    a = dict(a=Dev((4, 288), U8), a_sf=Dev((4, 3), U8), ids=Dev((4, 2), I32), weights=Dev((4, 2), F32),
             w13=Dev((5 * 6 * 8704,), U8), w2=Dev((5 * 3 * 8704,), U8), I=96, out=Dev((4, 288), B16),
             ws=Dev((1 << 20,), U8), err_flag=Dev((1,), I32))
    return mxq.mxq_experts_a8w4(**{**a, **kw})


CALLS = {
    norm: dict(x=B16, weight=B16, residual=B16, residual_out=B16, y=B16, q=U8, sc=U8),
    route: dict(logits=F32, bias=F32, ids=I32, weights=F32),
    prepare: dict(w=U8, w_e8m0=U8, out=U8),
    linear: dict(a=U8, a_sf=U8, w4=U8, out=B16),
    experts: dict(a=U8, a_sf=U8, ids=I32, weights=F32, w13=U8, w2=U8, out=B16, ws=U8, err_flag=I32),
}


@pytest.mark.parametrize("call", CALLS)
def test_good_calls_reach_the_library(lib, call):
    call()
    assert len(lib.calls) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS.items() for n in names])
def test_tensors_that_are_refused(lib, call, name):
    dtype = CALLS[call][name]
    shape = {"x": (4, 256), "weight": (256,), "residual": (4, 256), "residual_out": (4, 256), "y": (4, 256),
             "q": (4, 256), "sc": (4, 2), "logits": (4, 64), "bias": (64,), "ids": (4, 6) if call is route else (4, 2),
             "weights": (4, 6) if call is route else (4, 2), "w": (2, 128, 64), "w_e8m0": (2, 128, 4),
             "out": {prepare: (2 * 8704,), linear: (4, 128), experts: (4, 288)}.get(call), "a": (4, 288),
             "a_sf": (4, 3), "w4": (3 * 8704,), "w13": (5 * 6 * 8704,), "w2": (5 * 3 * 8704,), "ws": (1 << 20,),
             "err_flag": (1,)}[name]
    bad = [Dev(shape, dtype, device=-1), Dev(shape, dtype, device=1), Dev(shape, dtype, contiguous=False),
           Dev(shape, torch.float64)]
    if name not in ("ws", "x", "logits", "w", "a"):
        bad.append(Dev((*shape[:-1], shape[-1] + 1) if name != "err_flag" else (0,), dtype))
    for t in bad:
        with pytest.raises(mxq.MxqError):
            call(**{name: t})
    assert not lib.calls


def test_other_refusals(lib):
    with pytest.raises(mxq.MxqError):
        norm(residual=None)  # residual_out without it
    with pytest.raises(mxq.MxqError):
        norm(x=Dev((), B16))
    for bad in (dict(scoring="tanh"), dict(k=0), dict(k=-3)):
        with pytest.raises(mxq.MxqError):
            route(**bad)
    with pytest.raises(mxq.MxqError):
        prepare(w=Dev((128,), U8))
    for bad in (dict(I=90), dict(N=24), dict(w2=Dev((100,), U8))):
        with pytest.raises(mxq.MxqError):
            experts(**bad)
    assert not lib.calls


def test_sizes_beyond_32_bits(lib):
    """Sizes that 32-bit arguments would cut down to good ones."""
    over = 1 << 32
    for call, bad in ((norm, dict(x=Dev((4, over + 256), B16))), (route, dict(k=over + 6)), (route, dict(groups=over + 1)),
                      (route, dict(logits=Dev((4, over + 64), F32))), (linear, dict(N=over + 128)),
                      (experts, dict(I=over + 96)), (experts, dict(N=over + 288)),
                      (prepare, dict(w=Dev((over + 2, 128, 64), U8)))):
        with pytest.raises(mxq.MxqError, match="32 bits"):
            call(**bad)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_w4_bytes(1, over + 16, 32)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_experts_workspace_bytes(1, 1, 1, 32, over + 32, 16)
    assert not lib.calls


def test_the_current_device_is_another(lib, monkeypatch):
    monkeypatch.setattr(mxq, "_current_device", lambda: 1)
    for call in CALLS:
        with pytest.raises(mxq.MxqError):
            call()
    assert not lib.calls


class Recorder:
    """Stands in for torch in the binding: tensors on the CPU, with the stream current at their allocation."""

    def __init__(self):
        self.now, self.allocs = "current", []
        self.cuda = types.SimpleNamespace(stream=self.stream)

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
        return torch.empty(t.shape, dtype=t.dtype)


ALLOCS = [(lambda **k: norm(residual_out=None, y=None, q=None, sc=None, **k), 4),
          (lambda **k: norm(residual=None, residual_out=None, y=None, want_y=False, q=None, sc=None, **k), 2),
          (lambda **k: route(ids=None, weights=None, **k), 2), (lambda **k: prepare(out=None, **k), 1),
          (lambda **k: linear(out=None, **k), 1), (lambda **k: experts(out=None, ws=None, **k), 2)]


@pytest.mark.parametrize("call,n", ALLOCS)
def test_allocations_belong_to_the_stream(lib, monkeypatch, call, n):
    rec = Recorder()
    monkeypatch.setattr(mxq, "torch", rec)
    call(stream=types.SimpleNamespace(name="side", cuda_stream=7))
    assert rec.allocs == ["side"] * n and rec.now == "current"
    rec.allocs.clear()
    call()
    assert rec.allocs == ["current"] * n


def test_the_quick_way_is_that_of_this_torch(monkeypatch, tmp_path):
    """A module built against another torch is not loaded; the calls then go through ctypes."""
    from importlib.machinery import EXTENSION_SUFFIXES

    (tmp_path / f"mxq_fastcall-0.0{EXTENSION_SUFFIXES[0]}").write_bytes(b"not to be loaded")
    monkeypatch.setattr(mxq, "HERE", str(tmp_path))
    monkeypatch.setattr(mxq, "_fast", None)
    assert mxq._fastcall() is False
    assert build.fastcall_path(torch.__version__).endswith(f"mxq_fastcall-{torch.__version__}{EXTENSION_SUFFIXES[0]}")


def test_the_quick_way_leaves_the_rest():
    """On the CPU nothing is the common case: each function answers None, and the errors are the Python code's."""
    build.build()
    f = mxq._fastcall()
    if not f:
        pytest.skip("mxq_fastcall was not built")
    x, u = torch.zeros((4, 256), dtype=B16), torch.zeros((4, 256), dtype=U8)
    for call in (lambda: f.norm(x, None, 1e-6, None, True, True), lambda: f.norm(None, None, 1e-6, None, True, True),
                 lambda: f.norm(Dev((4, 256), B16), None, 1e-6, None, True, True), lambda: f.norm(x),
                 lambda: f.route(x, 2, 0, None, 1, 1, 2, True, 1.0), lambda: f.route("x", 2, 0, None, 1, 1, 2, True, 1.0),
                 lambda: f.linear(u, u, u, 16), lambda: f.linear(u), lambda: f.experts(u, u, u, u, u, u, 32, 32)):
        assert call() is None
    for call in (lambda: mxq.mxq_add_rms_norm(x), lambda: mxq.mxq_route(x, 2), lambda: mxq.mxq_linear_a8w4(u, u, u, 16),
                 lambda: mxq.mxq_experts_a8w4(u, u, u.int(), u.float(), u, u, 32)):
        with pytest.raises(mxq.MxqError):
            call()
    with pytest.raises(TypeError):
        f.bind(1)
    with pytest.raises(ValueError):
        f.bind(0, 0, 0, 0, 0, 0)
