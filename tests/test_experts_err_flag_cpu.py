"""mxq_experts_a8w4: an error word inside any other buffer of the call is refused (its bit would change that buffer)."""

import pytest
import torch

from test_ffn_abi_cpu import C, L, Q, R, S, W, X, Y, experts  # noqa: F401  (L: the library's fixture)

E, K, I, N, T, k = 16, 576, 288, 1024, 4, 8
BLOCK = 8704
SIZES = {X: T * K, R: T * 5, S: T * k * 4, W: T * k * 4, Y: 2 * E * 3 * 5 * BLOCK, Q: E * 8 * 3 * BLOCK, C: T * N * 2}


@pytest.mark.parametrize("base", list(SIZES))
def test_error_words_in_other_buffers(L, base):  # noqa: F811
    n = SIZES[base]
    for err in (base, base + n // 2 & ~3, base + (n - 1 & ~3)):
        assert experts(L, err=err) == 2, (base, err)
    if not torch.cuda.is_available():
        for err in (base - 4, base + (n + 3 & ~3)):
            assert experts(L, err=err) == 7, (base, err)
