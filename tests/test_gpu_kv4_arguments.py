"""Plans of verify_kv4 are kept by the values of a call's arguments, whatever objects carry them."""
import numpy as np
import pytest

from _helpers import bf16_dev, to_dev
from speculative_decode_mla_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def test_arguments_held_in_tensors_are_read_at_every_call():
    """0-d tensors and numpy scalars as max_seq_len, scale, hint and splits, changed in place between two calls."""
    import torch
    import oracle
    import speculative_decode_mla_gb300 as m
    p = W.custom_problem([600, 35], 3, 4, seed=91)
    x = W.normal_bf16(92, p.num_slots * 576).reshape(p.num_slots, 576)
    pool = to_dev(oracle.kv4_quantise(x))
    dev = (bf16_dev(p.q), pool, to_dev(p.slot_table))
    parents = to_dev(p.tree_parent)
    most, scale, hint, splits = torch.tensor(300), torch.tensor(0.05), torch.tensor(300), torch.tensor(2)
    short = to_dev(np.array([300, 20], np.int32))
    a = m.verify_kv4(*dev, short, parents, max_seq_len=most, softmax_scale=scale, total_tokens_hint=hint, num_splits=splits)
    b = m.verify_kv4(*dev, short, parents, max_seq_len=300, softmax_scale=float(scale), total_tokens_hint=300, num_splits=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    most.fill_(600)
    scale.fill_(0.0721)
    hint.fill_(700)
    splits.fill_(5)
    full = to_dev(p.seq_lens)
    a = m.verify_kv4(*dev, full, parents, max_seq_len=most, softmax_scale=scale, total_tokens_hint=hint, num_splits=splits)
    b = m.verify_kv4(*dev, full, parents, max_seq_len=np.int32(600), softmax_scale=float(scale), total_tokens_hint=700, num_splits=5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
