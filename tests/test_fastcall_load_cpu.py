"""A module of the binding's quick way in that does not load is an error at each call, not at the first alone."""

from importlib.machinery import EXTENSION_SUFFIXES

import pytest
import torch

import mxfp8_block_scaled_inv_gb300 as mxq
from mxfp8_block_scaled_inv_gb300 import build


def test_a_module_that_does_not_load(monkeypatch, tmp_path):
    build.build()
    (tmp_path / f"mxq_fastcall-{torch.__version__}{EXTENSION_SUFFIXES[0]}").write_bytes(b"no library")
    monkeypatch.setattr(mxq, "HERE", str(tmp_path))
    monkeypatch.setattr(mxq, "_fast", None)
    for _ in range(3):
        with pytest.raises(mxq.MxqLibraryError):
            mxq._fastcall()
    u = torch.zeros((4, 256), dtype=torch.uint8)
    with pytest.raises(mxq.MxqLibraryError):
        mxq.mxq_linear_a8w4(u, u, u, 16)
