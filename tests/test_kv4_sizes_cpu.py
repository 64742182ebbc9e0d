"""Sizes of attention over the 4-bit cache that its checks have to see through."""
from __future__ import annotations

import pytest
import torch

import int4_quantized_gemm_b200 as qg
from test_kv4_args_cpu import F, I, R, U, attend, cache


@pytest.mark.parametrize("page", [16, 64, 65536])
@pytest.mark.parametrize("power", [31, 32, 48, 58, 60, 62])
def test_tables_whose_tokens_leave_64_bits_are_refused(page, power):
    """max_pages * page_size may be 0 in 64 bits."""
    assert attend(c=cache(page=page), pages=1 << power, ld=1 << power) == U


def test_sequences_next_to_2_to_the_31_are_refused():
    """The end of their last step would not fit in 32 bits."""
    for page, pages in ((16, (1 << 27) - 1), (16, (1 << 27) - 7), (48, (1 << 31) // 48), (64, (1 << 25) - 1)):
        assert attend(c=cache(page=page, heads=1), B=1, T=1, Hq=1, pages=pages, ld=pages) == U
    if not torch.cuda.is_available():                 # (a device would run the call, whose pointers are made up)
        assert attend(c=cache(page=16, heads=1), B=1, T=1, Hq=1, pages=(1 << 27) - 8, ld=1 << 27) == qg.QG_ERR_NO_DEVICE


def test_query_tokens_of_no_sequence_are_refused():
    """Nothing would write their outputs; with starts they lie behind the last sequence and are left alone."""
    assert attend(B=0, T=2) == I
    assert attend(B=0, T=2, starts=F) == 0 and attend(B=0, T=0) == 0


def test_no_workspace_for_calls_that_are_refused():
    f = R.qg_attention_kv4_workspace_size
    assert f(1, 1 << 40, 1 << 40, 1, 64, 0) == 0 and f(4097, 4097, 4, 2, 64, 0) == 0 and f(1, 1 << 31, 1, 1, 64, 1) == 0
    assert f(2, 1 << 33, 1 << 31, 1, 64, 1) == 0
