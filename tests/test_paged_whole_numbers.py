"""Numbers that do not fit the C entry points' 32-bit arguments are refused, not cut off:
2**32 + 1 new tokens are not one."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
from exact_attention_blackwell_gb300 import build as fa_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("n", [2**32 + 1, 2**31, -(2**31) - 1, 2**64 + 16, -(2**32) + 16])
def test_numbers_past_32_bits(n):
    with pytest.raises(ValueError, match="max_new must fit 32 bits"):
        fa.attention_fwd_paged(bf(5, 4, 64), bf(9, 16, 2, 64), bf(9, 16, 2, 64), i32(3, 4), i32(3), i32(4), n)
    with pytest.raises(ValueError, match="page_size must fit 32 bits"):
        fa.cache_fork(i32(9), i32(3, 4), i32(3), i32(3), n)


def test_numbers_that_fit_go_on_to_the_next_check():
    for n in (1, 2**31 - 1, -(2**31)):
        with pytest.raises(ValueError, match="CUDA"):
            fa.attention_fwd_paged(bf(5, 4, 64), bf(9, 16, 2, 64), bf(9, 16, 2, 64), i32(3, 4), i32(3), i32(4), n)
        with pytest.raises(ValueError, match="CUDA"):
            fa.cache_fork(i32(9), i32(3, 4), i32(3), i32(3), n)
