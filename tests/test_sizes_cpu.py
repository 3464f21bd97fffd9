"""Sizes beyond the library's 32-bit arguments are refused, not cut off."""

import pytest

BIG = 2 ** 32 + 4


def test_workspace_sizes():
    from bit_quantized_moe_token_amd import moeq
    assert moeq.linear_i8_workspace_size(4, 64) == 4 * (128 + 4)
    for f in (moeq.linear_i8_workspace_size, moeq.block_norm_grad_workspace_size):
        for bad in ((BIG, 64), (4, BIG + 60), (2 ** 31, 64)):
            with pytest.raises(ValueError):
                f(*bad)
        with pytest.raises(moeq.MoeqError):
            f(2 ** 31 - 1, 2 ** 31 - 1)
