"""Limits of mla_prompt_attn's scalar arguments (no GPU)."""
import ctypes

import pytest

import speculative_decode_mla_gb300 as m
from speculative_decode_mla_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m.load_library()


@pytest.mark.parametrize("scale,want", [(2.0 ** 127, 0), (1e38, 0), (2.0 ** -149, 0), (1.8e38, -1), (3.4e38, -1), (-1.0, -1), (-0.0, -1)])
def test_scales(lib, scale, want):
    """A scale whose product with log2 e is no float32 number is refused."""
    d = m.PromptDesc(num_seqs=1, num_heads=2, num_kv_heads=2, max_q_len=5, max_k_len=5, causal=1, softmax_scale=scale, num_q=5, num_k=5,
                     q_token_stride=384, q_head_stride=192, k_token_stride=256, k_head_stride=128, k_rope_token_stride=64, v_token_stride=256,
                     v_head_stride=128)
    assert lib.mla_prompt_plan(ctypes.byref(d), 152, ctypes.byref(m.PromptPlan())) == want


@pytest.mark.parametrize("seqs,want", [(1 << 30, 0), ((1 << 30) + 1, -2), (2 ** 31 - 1, -2)])
def test_numbers_of_sequences(lib, seqs, want):
    """The kernels count sequences in 32 bits, in steps of up to 1024 behind the last."""
    d = m.PromptDesc(num_seqs=seqs, num_heads=1, num_kv_heads=1, max_q_len=1, max_k_len=1, causal=1, softmax_scale=1.0, num_q=1, num_k=1)
    assert lib.mla_prompt_plan(ctypes.byref(d), 152, ctypes.byref(m.PromptPlan())) == want
