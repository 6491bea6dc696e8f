"""Limits of the operators around the decode step, on the CPU: sizes and numbers that the C entry points and the binding have
to refuse."""

import ctypes

import pytest
import torch

import block_sparse_attention_attngate_b200 as S
from block_sparse_attention_attngate_b200 import seer
from test_serving_abi import plan, reaches_cuda, release, said

lib = seer._lib


# ---------------------------------------------------------------- pages
@pytest.mark.parametrize("over", [1, 255, 65535, (1 << 17) - 1])
def test_page_kernels_count_in_31_bits(over):
    """The kernels step 32-bit indexes by up to 65536 elements past the last one: sizes that near 2^31 are refused."""
    most = 2 ** 31 - 2 ** 17
    assert plan(room=most + over) == 2 and said("max_tokens")
    for call in (plan, release):
        assert call(page=1, pages=most + over) == 2 and said("num_pages")
    reaches_cuda(lambda: plan(room=most))
    reaches_cuda(lambda: plan(page=1, pages=most))
    reaches_cuda(lambda: release(page=1, pages=most))
