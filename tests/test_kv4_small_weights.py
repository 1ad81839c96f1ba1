"""What the GPU test of many small weights beside a large one relies on, checked on the oracle (no GPU)."""
import numpy as np

import oracle
from speculative_decode_mla_gb300 import workloads as W


def test_twenty_thousand_small_weights_add_up_beside_a_large_one():
    """Keys without RoPE dims but for one, whose score is 16 * 9 / sqrt(192): every other weight is tiny next to its weight, and
    together they are a sizeable share."""
    p = W.custom_problem([20000], 1, 2, seed=45, pool_slack=7, stride_pad=3)
    x = W.bf16_bits_to_f32(W.normal_bf16(1045, p.num_slots * 576)).reshape(p.num_slots, 576).copy()
    x[:, 512:] = 0
    x[p.slot_table[0, 777], 512] = 9
    q = np.zeros((1, 2, 576), np.float32)
    q[:, :, 512] = 16
    q = W.f32_to_bf16_bits(q).reshape(p.q.shape)
    bits = oracle.kv4_bf16(oracle.kv4_quantise(W.f32_to_bf16_bits(x)))
    _, lse = oracle.verify(p.seq_lens, p.slot_table, p.tree_parent, q, bits, num_heads=2, scale=W.SOFTMAX_SCALE)
    large, small = np.exp(16 * 9 * W.SOFTMAX_SCALE - lse), np.exp(0 - lse)
    assert (small < 2.0 ** -14 * large).all() and (0.3 < 20000 * small).all() and (20000 * small < 0.5).all()
    assert np.allclose(large + 20000 * small, 1, atol=1e-9)
