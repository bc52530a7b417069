"""Sizes at the ends of what 32 bits count, without a GPU: refused before any
launch."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import attention as A

SHAPE = 2


def heads():
    return ctypes.byref(A.Heads(4096, 256, 64))


@pytest.mark.parametrize("total_k", [2 ** 31 - 1, 2 ** 31 - 127])
def test_keys_whose_last_block_passes_31_bits(native, total_k):
    assert A.load().moe_attention_prompt(heads(), heads(), heads(), 16, 16, 1, 4, total_k, 4, 2, 64, 0, 0.1, heads(), None,
                                         None) == SHAPE


@pytest.mark.parametrize("tokens,heads", [(2 ** 31, 1), (2 ** 32 + 5, 1), (2, 2 ** 31)])
def test_tensors_of_more_tokens_than_an_int_holds(tokens, heads):
    """Their low 32 bits would be another size. (Broadcast rows: no memory is needed.)"""
    rows = torch.zeros((1, 1, 8), dtype=torch.bfloat16).expand(tokens, heads, 8)
    with pytest.raises(ValueError, match="less than 2"):
        A._heads("q", rows, torch.bfloat16, -1)
    _, shape = A._heads("q", rows[:2, :1], torch.bfloat16, -1)
    assert tuple(shape) == (2, 1, 8)


@pytest.mark.parametrize("shape", [(0, 2, 8), (0, 1, 64)])
def test_strides_of_tensors_without_tokens_say_nothing(shape):
    """A step in which no sequence grows: torch gives empty tensors any strides."""
    rows = torch.zeros(0, dtype=torch.bfloat16)[:, None, None].expand(shape)
    assert rows.is_contiguous() and rows.stride(2) == 0
    _, got = A._heads("k", rows, torch.bfloat16, -1)
    assert tuple(got) == shape
