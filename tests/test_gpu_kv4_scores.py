"""Attention over the 4-bit pool when finite keys and queries give very large scores: the key with the largest score takes
all the weight, keys with equal scores share it, and nothing overflows on the way."""
import numpy as np
import pytest

import oracle
from _helpers import bf16_dev, to_dev
from speculative_decode_mla_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()


KERNELS = {"tcgen05": ([700, 90], 3, 16, 0, 0), "tcgen05 in one part": ([700, 90], 3, 16, 0, 1), "few rows": ([700, 90] * 9, 2, 6, 2, 0),
           "simt": ([700, 90], 3, 16, 1, 0)}


def check(kernel, q_size, k_size, scale=W.SOFTMAX_SCALE):
    """Queries are +-1.5 q_size in the first RoPE dim and zero elsewhere. Of each sequence's keys two have 1.25 k_size there
    (positions in different tiles), one has -1.5 k_size, all others little, so every score is one product and the weights are
    exactly 1/2 and 1/2 for the one sign and 1 for the other. The pool's values have 6 bits, so a half of a sum of two of them
    has at most 11 where their scales are within a factor of 2^4 (they are: one row's latents are a copy of the other's with
    other signs), and every step of the way to the fp32 output is exact. lse: the scale, log2(e) and ln(2) in fp32, the two
    products that put them together, the score times them, the maximum less 7 and plus the sum's logarithm, the product with
    ln(2) and the merge of the parts: ten roundings of at most 2^-24 each."""
    import torch
    import speculative_decode_mla_gb300 as m
    lens, T, H, number, splits = KERNELS[kernel]
    p = W.custom_problem(lens, T, H, seed=95, pool_slack=5)
    x = W.bf16_bits_to_f32(W.normal_bf16(96, p.num_slots * 576)).reshape(p.num_slots, 576).copy()
    x[:, 512:] = 0
    want_o, want_l = np.zeros((p.B, T * H, 512)), np.zeros((p.B, T * H))
    sign = np.where(np.arange(T * H) % 2 == 0, 1.0, -1.0)
    for b in range(p.B):
        j, k, n = (int(p.slot_table[b, t]) for t in (10, p.seq_lens[b] - 1, 33))
        x[k, :512] = x[j, :512] * np.where(np.arange(512) % 3 == 0, -1, 1)
        x[j, 512] = x[k, 512] = np.float32(1.25 * k_size)
        x[n, 512] = np.float32(-1.5 * k_size)
    rows = oracle.kv4_quantise(W.f32_to_bf16_bits(x))
    values = oracle.kv4_values(rows)
    for b in range(p.B):
        j, k, n = (int(p.slot_table[b, t]) for t in (10, p.seq_lens[b] - 1, 33))
        want_o[b] = np.where(sign[:, None] > 0, (values[j, :512] + values[k, :512]) / 2, values[n, :512])
        want_l[b] = np.where(sign > 0, 1.5 * 1.25 * q_size * k_size * scale + np.log(2), 1.5 * 1.5 * q_size * k_size * scale)
    q = np.zeros((p.B, T * H, 576), dtype=np.float32)
    q[:, :, 512] = sign * np.float32(1.5 * q_size)
    q = W.f32_to_bf16_bits(q).reshape(p.q.shape)
    d = m.make_desc(p.B, T, H, p.num_slots, p.slot_table.shape[1], p.max_seq_len, flags=m.MLA_FLAG_SIMT if number == 1 else 0)
    assert m.kv4_plan(d, 152).kernel == number
    out, lse = m.verify_kv4(bf16_dev(q), to_dev(rows), to_dev(p.slot_table), to_dev(p.seq_lens), to_dev(p.tree_parent),
                            max_seq_len=p.max_seq_len, out_dtype=m.MLA_DTYPE_F32, num_splits=splits, softmax_scale=scale,
                            flags=m.MLA_FLAG_SIMT if number == 1 else None)
    torch.cuda.synchronize()
    o, l = out.cpu().numpy().reshape(want_o.shape), lse.cpu().numpy().reshape(want_l.shape).astype(np.float64)
    assert np.isfinite(l).all(), f"{np.isfinite(l).mean():.2f} of the lse values are finite"
    assert (np.abs(l / want_l - 1) <= 10 * 2.0 ** -24).all(), f"lse: {np.abs(l / want_l - 1).max():.2e} relative"
    assert np.array_equal(o, want_o), f"out: {(o != want_o).mean():.2f} of the values differ"


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("power", [16, 24, 27, 28, 29, 33, 48, 80, 100])
def test_scores_far_beyond_the_weights_range(kernel, power):
    check(kernel, 1.0, 2.0 ** power)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("q_size,k_size", [(1.0, 2.0 ** 113), (1.0, 2.0 ** 125), (2.0 ** -20, 2.0 ** 127), (2.0 ** -100, 2.0 ** 127),
                                           (2.0 ** 60, 2.0 ** 64), (2.0 ** 126, 1.0)])
def test_keys_and_queries_up_to_the_types_largest(kernel, q_size, k_size):
    check(kernel, q_size, k_size)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("power", [-131, -127, -121, -100])
def test_the_smallest_queries_with_the_largest_keys(kernel, power):
    """Query rows from bf16's subnormals on against RoPE keys near its largest, so that the scores are ordinary. A weight and a part's
    output are rounded to fp16 (2^-11 each), the rest is fp32: a score is off by at most 576 * 2^-24 of the sum of its products'
    magnitudes (64 of at most 4 * 4 * 16 times the scale of 0.072: below 64 * 2^5), which moves the lse and, with the norm, weights
    by twice as much."""
    import torch
    import speculative_decode_mla_gb300 as m
    lens, T, H, number, splits = KERNELS[kernel]
    p = W.custom_problem(lens, T, H, seed=97, pool_slack=5)
    x = W.bf16_bits_to_f32(W.normal_bf16(98, p.num_slots * 576)).reshape(p.num_slots, 576).copy()
    k_size, q_size = (2.0 ** 124, 2.0 ** power) if power < -118 else (2.0 ** (4 - power), 2.0 ** power)
    x[:, 512:] = np.clip(x[:, 512:], -4, 4) * np.float32(k_size)
    q = W.bf16_bits_to_f32(p.q).copy()
    q = W.f32_to_bf16_bits(np.clip(q, -4, 4) * np.float32(q_size)).reshape(p.q.shape)
    rows = oracle.kv4_quantise(W.f32_to_bf16_bits(x))
    o, l = oracle.verify(p.seq_lens, p.slot_table, p.tree_parent, q, oracle.kv4_bf16(rows), num_heads=H, scale=W.SOFTMAX_SCALE)
    out, lse = m.verify_kv4(bf16_dev(q), to_dev(rows), to_dev(p.slot_table), to_dev(p.seq_lens), to_dev(p.tree_parent),
                            max_seq_len=p.max_seq_len, out_dtype=m.MLA_DTYPE_F32, num_splits=splits,
                            flags=m.MLA_FLAG_SIMT if number == 1 else None)
    torch.cuda.synchronize()
    d_score = 576 * 2.0 ** -24 * 64 * 2.0 ** 5
    top = np.abs(oracle.kv4_values(rows)[:, :512]).max()
    assert np.abs(lse.cpu().numpy().reshape(-1) - l.reshape(-1)).max() <= d_score
    assert np.abs(out.cpu().numpy().reshape(-1, 512) - o.reshape(-1, 512)).max() <= (2 * 2.0 ** -11 + 2 * d_score) * top
