"""The workspace that mxq_attn_workspace_bytes names is enough for the call, with
and without q_start: the plan follows from what the query takes.  Without a
device a call whose arguments are accepted returns MXQ_ERR_CUDA."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p(1 << 20)
Q = ctypes.c_void_p(1 << 50)


@pytest.fixture(scope="module")
def L():
    from mxfp8_block_scaled_inv_gb300 import build as B

    B.build()
    import mxfp8_block_scaled_inv_gb300 as mxq

    return mxq.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("H,D", [(1, 64), (12, 192), (32, 512), (96, 512), (128, 512), (128, 128)])
def test_queried_size_is_accepted(L, H, D):
    """Batches of one token each (T == B) and of several, capacities of 64 to 32768 keys, windows."""
    some = 0
    for B in [*range(1, 40, 3), *range(40, 330, 7), 1500]:
        for T in (B, 2 * B):
            for pages in (1, 5, 16, 100, 512):
                for window in (0, 300):
                    need = L.mxq_attn_workspace_bytes(T, B, H, D, pages, 64, window, 4)
                    some += need > 0
                    for q_start in (P, None) if T == B else (P,):
                        st = L.mxq_attn(P, T, H, D, q_start, P, B, P, pages, 64, P, 4096, 1, None, None, window, 4,
                                        0.1, Q, None, None, P if need else None, need, None)
                        assert st == 7, (B, T, pages, window, q_start, need, L.mxq_last_error())
    assert some > 100


def test_wait_bound_is_a_plain_setting(L):
    assert L.mxq_debug_set_attn_wait(5000) == 2_000_000_000
    assert L.mxq_debug_set_attn_wait(3_000_000_000) == 5000  # above the most: the default
    assert L.mxq_debug_set_attn_wait(0) == 2_000_000_000
