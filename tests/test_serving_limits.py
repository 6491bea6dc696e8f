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


# ---------------------------------------------------------------- whole numbers that 32 bits do not hold
def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def half(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def flat(t):
    return S.KVCache(S.KVDesc(0, 0, t.stride(0), t.stride(1), t.stride(2), t.shape[2], 0, None, 0), (t,), t.dtype)


def paged(t, table):
    return S.KVCache(S.KVDesc(1, 0, t.stride(0), t.stride(1), t.stride(2), 0, t.shape[0], None, 8), (t, table), t.dtype)


PLAN = dict(page_size=16, seqlens=i32(1), new_tokens=i32(1), block_table=i32(1, 8), free_list=i32(64), free_count=i32(1),
            cu_tokens=i32(2), slot_map=i32(32), positions=i32(32))
RELEASE = dict(page_size=16, seqlens=i32(1), finished=i32(1), block_table=i32(1, 8), free_list=i32(64), free_count=i32(1))
ROPE = dict(q=half(3, 4, 128), k=half(3, 2, 128), positions=i32(3), q_out=half(3, 4, 128))
GRAD = dict(dq_out=half(3, 4, 128), dk_out=None, q=half(3, 4, 128), k=None, positions=i32(3), dq=half(3, 4, 128), dk=None)
DENSE = dict(q=half(2, 8, 128), k=flat(half(2, 2, 64, 128)), v=flat(half(2, 2, 64, 128)), seqlens=i32(2),
             out=half(2, 8, 128), workspace=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("fn,good,name", [(S.page_plan, PLAN, "page_size"), (S.page_release, RELEASE, "page_size"),
                                          (S.qk_norm_rope, ROPE, "rope_dim"), (S.qk_norm_rope_backward, GRAD, "rope_dim"),
                                          (S.dense_decode, DENSE, "window")])
def test_numbers_past_32_bits_are_refused(fn, good, name):
    """Handed on as 32-bit arguments they would be taken modulo 2^32."""
    for bad in (2 ** 32 + 16, 2 ** 31, -2 ** 31 - 1, -2 ** 32 + 16, 2 ** 70, 16.5, float("nan"), float("inf")):
        with pytest.raises(ValueError, match=name):
            fn(**{**good, name: bad})
    for fine in (16, 16.0, torch.tensor(16)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            fn(**{**good, name: fine})


def test_extents_past_32_bits_are_refused():
    """Tensors as wide as that (one element, repeated: nothing is allocated)."""
    wide = 2 ** 32 + 8
    for fn, good in ((S.page_plan, PLAN), (S.page_release, RELEASE)):
        for name, bad in (("block_table", i32(1, 1).expand(1, wide)), ("free_list", i32(1).expand(wide))):
            with pytest.raises(ValueError, match=name):
                fn(**{**good, name: bad})
    with pytest.raises(ValueError, match="slot_map"):
        S.page_plan(**{**PLAN, "slot_map": i32(1).expand(wide), "positions": i32(1).expand(wide)})
    with pytest.raises(ValueError, match="block table"):
        S.dense_decode(**{**DENSE, "k": paged(half(9, 2, 7, 128), i32(2, 1).expand(2, wide))})
    with pytest.raises(ValueError, match="page"):
        S.dense_decode(**{**DENSE, "k": paged(half(9, 2, 1, 128).expand(9, 2, wide, 128), i32(2, 8))})
    with pytest.raises(ValueError, match="k_cache"):
        S.qk_norm_rope(**{**ROPE, "k_cache": half(4, 2, 1, 128).expand(4, 2, wide, 128), "slot_map": i32(3)})
    rows = half(1, 4, 128).expand(wide, 4, 128)
    with pytest.raises(ValueError, match="tokens"):
        S.qk_norm_rope(rows, None, i32(1).expand(wide), rows)


def test_workspace_sizes_of_numbers_past_32_bits():
    for bad in (2 ** 32 + 128, 2 ** 31, 128.5):
        with pytest.raises(ValueError, match="head_dim"):
            S.norm_workspace_bytes(bad)
    good = dict(batch=1, num_q_heads=4, num_kv_heads=1, head_dim=64)
    for name in good:
        with pytest.raises(ValueError, match=name):
            S.dense_decode_workspace_bytes(**{**good, name: good[name] + 2 ** 32})


def test_softmax_scale_below_fp32_is_refused():
    """Rounded to fp32 it would be 0, which asks for 1 / sqrt(head_dim)."""
    for bad in (1e-46, -1e-300):
        with pytest.raises(ValueError, match="softmax_scale"):
            S.dense_decode(**DENSE, softmax_scale=bad)
    for fine in (0, 0.0, 2e-45, 1, 0.125):
        with pytest.raises(TypeError, match="CUDA tensor"):
            S.dense_decode(**DENSE, softmax_scale=fine)
