"""Pins of the prompt operators' definitions, their plans, and their refusals (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

import oracle
import speculative_decode_mla_gb300 as m
from speculative_decode_mla_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m.load_library()


# -------------------------------------------------------------------------------------- the definitions

def table(n, rng):
    a = rng.uniform(0, 2 * np.pi, (n, 32))
    return np.concatenate([np.cos(a), np.sin(a)], 1), a


@pytest.mark.parametrize("halves", [False, True])
def test_turning_keeps_lengths_and_adds_angles(halves):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(7, 3, 64))
    ta, a = table(7, rng)
    tb, b = table(7, rng)
    both = np.concatenate([np.cos(a + b), np.sin(a + b)], 1)
    y = oracle.turn(x, ta, halves)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    assert np.allclose(oracle.turn(y, tb, halves), oracle.turn(x, both, halves))
    quarter = np.concatenate([np.zeros((7, 32)), np.ones((7, 32))], 1)
    z = oracle.turn(x, quarter, halves)      # (x, y) -> (-y, x)
    if halves:
        assert np.allclose(z[..., :32], -x[..., 32:]) and np.allclose(z[..., 32:], x[..., :32])
    else:
        assert np.allclose(z[..., 0::2], -x[..., 1::2]) and np.allclose(z[..., 1::2], x[..., 0::2])


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    assert np.allclose(oracle.norm(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0), [[3 / 2.5, 8 / 2.5, 0, 0]])
    assert oracle.norm(x, None, 1.0) is x
    assert np.allclose(oracle.norm(x, np.ones(4), 6.25), x / math.sqrt(12.5))


def test_prompt_attention_by_hand():
    """Two sequences: three places of which the last two are queries, and one query without a key."""
    rng = np.random.default_rng(2)
    q, k, kr, v = rng.normal(size=(3, 2, 192)), rng.normal(size=(3, 1, 128)), rng.normal(size=(3, 64)), rng.normal(size=(3, 1, 128))
    out, lse, _, _ = oracle.prompt_attn(q, k, kr, v, [0, 2, 3], [0, 3, 3], causal=True, scale=0.3)
    s = [0.3 * (q[0, 1, :128] @ k[t, 0] + q[0, 1, 128:] @ kr[t]) for t in range(2)]     # the first query sees two keys
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[0, 1], w[0] * v[0, 0] + w[1] * v[1, 0]) and np.isclose(lse[0, 1], np.log(np.exp(s).sum()))
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()
    whole, _, _, _ = oracle.prompt_attn(q, k, kr, v, [0, 2, 3], [0, 3, 3], causal=False, scale=0.3)
    assert np.allclose(whole[1], out[1]) and not np.allclose(whole[0], out[0])


def test_expanded_and_absorbed_attention_agree():
    """Causal attention over expanded keys and values is attention over the latent rows with the expansion put into the queries
    and the outputs: the last query of a prompt against the verify oracle's single node."""
    rng = np.random.default_rng(3)
    n, heads = 9, 2
    from speculative_decode_mla_gb300 import workloads as W
    bits = W.normal_bf16(5, n * 576).reshape(n, 576)
    rows = W.bf16_bits_to_f32(bits).reshape(n, 576).astype(np.float64)
    wk, wv = rng.normal(size=(heads, 512, 128)) * 0.05, rng.normal(size=(heads, 512, 128)) * 0.05
    q = rng.normal(size=(n, heads, 192))
    k, v = np.einsum("td,hde->the", rows[:, :512], wk), np.einsum("td,hde->the", rows[:, :512], wv)
    out, lse, _, _ = oracle.prompt_attn(q, k, rows[:, 512:], v, [0, n], [0, n], causal=True, scale=0.1)
    absorbed = np.concatenate([np.einsum("he,hde->hd", q[-1, :, :128], wk), q[-1, :, 128:]], 1)
    s = absorbed @ rows.T * 0.1
    w = np.exp(s - s.max(1, keepdims=True))
    lat = w / w.sum(1, keepdims=True) @ rows[:, :512]
    assert np.allclose(np.einsum("hd,hde->he", lat, wv), out[-1])
    assert np.allclose(np.log(np.exp(s).sum(1)), lse[-1])


# ---------------------------------------------------------------------------------------------- plans

def prompt_desc(**kw):
    base = dict(num_seqs=1, num_heads=8, num_kv_heads=8, max_q_len=1000, max_k_len=1000, causal=1, out_dtype=0, flags=0, num_ctas=0,
                softmax_scale=0.07, num_q=1000, num_k=1000, q_token_stride=8 * 192, q_head_stride=192, k_token_stride=8 * 256,
                k_head_stride=256, k_rope_token_stride=576, v_token_stride=8 * 256, v_head_stride=256)
    base.update(kw)
    return m.PromptDesc(**base)


@pytest.mark.parametrize("kw", [dict(), dict(max_q_len=1, num_q=1, num_k=100000, max_k_len=100000), dict(num_seqs=4096, num_q=4096, max_q_len=1),
                                dict(num_q=1 << 20, num_k=1 << 20, max_q_len=1 << 20, max_k_len=1 << 20, num_heads=128, num_kv_heads=8),
                                dict(num_seqs=31, num_q=5000, num_k=77777, max_q_len=5000, max_k_len=70000), dict(num_ctas=7), dict(num_q=0, num_k=0),
                                dict(max_q_len=0), dict(max_k_len=0), dict(num_ctas=1024), dict(flags=2), dict(num_kv_heads=1), dict(num_heads=12, num_kv_heads=4),
                                dict(num_heads=256, num_kv_heads=1, num_q=300, max_q_len=1)])
def test_plans_cover_every_row(lib, kw):
    d = prompt_desc(**kw)
    p = m.prompt_plan(d, 152)
    group = d.num_heads // d.num_kv_heads
    if d.flags & m.MLA_FLAG_SIMT:
        assert p.kernel == 1 and p.ctas == d.num_q * d.num_heads and not p.listed and not p.shared and p.workspace_bytes == 0
    else:
        assert p.pack == (group if group in (1, 2, 4, 8, 16, 32, 64, 128) else 1)
        most = min(d.max_q_len, d.num_q)
        assert p.kernel == 0 and p.rows_per_unit == (128 if most * p.pack <= 128 else 256) and p.listed == (d.num_seqs > 1 and not p.shared)
        entries = min(d.num_seqs * -(-most * p.pack // p.rows_per_unit), d.num_q * p.pack // p.rows_per_unit + d.num_seqs)
        units = entries * d.num_heads // p.pack
        assert p.ctas == ((d.num_ctas or 152) if p.shared else units)
        assert p.shared == (units > 0 and (d.num_ctas > 0 or (units < 4 * 152 and min(d.max_k_len, d.num_k) > 4 * 128)))
        need = p.ctas * 2 * p.rows_per_unit * (512 + 4) + 32 * p.ctas if p.shared else 0
        assert p.workspace_bytes >= need + (8 * entries if p.listed else 0)
    assert bytes(p) == bytes(m.prompt_plan(d, 152))


@pytest.mark.parametrize("bad", [dict(num_seqs=0), dict(num_heads=0), dict(num_kv_heads=3), dict(num_kv_heads=0), dict(max_q_len=-1),
                                 dict(max_k_len=-1), dict(causal=2), dict(out_dtype=2), dict(flags=4), dict(num_ctas=-1),
                                 dict(num_ctas=1025), dict(softmax_scale=0.0), dict(softmax_scale=float("nan")),
                                 dict(softmax_scale=float("inf")), dict(num_q=-1), dict(num_k=-1), dict(q_token_stride=1537),
                                 dict(q_head_stride=0), dict(k_token_stride=4), dict(k_head_stride=-256), dict(k_rope_token_stride=0),
                                 dict(v_token_stride=1 << 39), dict(v_head_stride=12), dict(num_q=(1 << 30) + 1), dict(num_q=1 << 28), dict(num_k=1 << 31)])
def test_plan_refuses(lib, bad):
    d = prompt_desc(**bad)
    assert lib.mla_prompt_plan(ctypes.byref(d), 152, ctypes.byref(m.PromptPlan())) in (-1, -2)
    assert lib.mla_prompt_workspace_size(ctypes.byref(d), ctypes.byref(ctypes.c_size_t())) in (-1, -2)


def test_strides_of_single_elements_are_not_looked_at(lib):
    d = prompt_desc(num_heads=1, num_kv_heads=1, num_q=1, num_k=1, q_token_stride=3, q_head_stride=5, k_token_stride=1, k_head_stride=0,
                    k_rope_token_stride=1, v_token_stride=7, v_head_stride=2)
    assert m.prompt_plan(d, 152).ctas == 1


def test_attn_refuses_bad_pointers(lib):
    d, x = prompt_desc(), 1 << 20
    good = dict(q=x, k=x, kr=x, v=x, cu_q=x, cu_k=x, out=x, lse=x, ws=x)

    def call(desc=d, **kw):
        a = {**good, **kw}
        return lib.mla_prompt_attn(ctypes.byref(desc), a["q"] or None, a["k"] or None, a["kr"] or None, a["v"] or None, a["cu_q"] or None,
                                   a["cu_k"] or None, a["out"] or None, a["lse"] or None, a["ws"] or None, 1 << 30, None, None)

    for name in ("q", "k", "kr", "v", "cu_q", "cu_k", "out", "lse"):
        assert call(**{name: 0}) == -1, name
    for name in ("q", "k", "kr", "v", "out"):
        assert call(**{name: x + 8}) == -1, name
    for name in ("cu_q", "cu_k", "lse"):
        assert call(**{name: x + 2}) == -1, name
    assert call(ws=x + 16) == -1
    assert call(desc=prompt_desc(flags=m.MLA_FLAG_DEBUG_CHECKS)) == -1     # needs dev_status
    assert call(desc=prompt_desc(num_heads=0)) == -1


def rope_desc(**kw):
    base = dict(num_rows=10, row_stride=576, num_slots=100, q_token_stride=8 * 192, q_head_stride=192, q_out_token_stride=8 * 192,
                q_out_head_stride=192, pool_format=m.MLA_POOL_BF16, num_heads=8, head_dim=192, num_positions=50, pairs=0, eps=1e-6)
    base.update(kw)
    return m.RopeDesc(**base)


X = 1 << 20


@pytest.mark.parametrize("desc,args,want", [
    (dict(num_rows=-1), {}, -1), (dict(row_stride=568), {}, -1), (dict(row_stride=577), {}, -1), (dict(num_slots=0), {}, -1),
    (dict(num_slots=1 << 31), {}, -1), (dict(pool_format=3), {}, -1), (dict(num_heads=0), {}, -1), (dict(head_dim=56), {}, -1),
    (dict(head_dim=100), {}, -1), (dict(head_dim=264, q_out_head_stride=264, q_out_token_stride=8 * 264), {}, -2),
    (dict(num_positions=0), {}, -1), (dict(pairs=2), {}, -1),
    (dict(eps=-1.0), {}, -1), (dict(eps=float("nan")), {}, -1), (dict(q_token_stride=3), {}, -1), (dict(q_head_stride=-8), {}, -1),
    (dict(q_out_head_stride=184), {}, -1), (dict(q_out_token_stride=0), {}, -1), (dict(q_out_token_stride=7 * 192), {}, -1), (dict(num_heads=1 << 30), {}, -2),
    ({}, dict(rows=X + 8), -1), ({}, dict(weight=X + 2), -1), ({}, dict(q=X + 8), -1), ({}, dict(q_weight=X + 8), -1),
    ({}, dict(positions=0), -1), ({}, dict(positions=X + 2), -1), ({}, dict(cos_sin=0), -1), ({}, dict(cos_sin=X + 4), -1),
    ({}, dict(slot_map=0), -1), ({}, dict(slot_map=X + 2), -1), ({}, dict(pool=0), -1), ({}, dict(pool=X + 8), -1),
    (dict(pool_format=m.MLA_POOL_KV4), dict(pool=X + 16), -1), ({}, dict(rows_out=X + 8), -1), ({}, dict(q_out=0), -1),
    ({}, dict(q_out=X + 8), -1), ({}, dict(debug=1), -1), ({}, dict(rows=0), -1), ({}, dict(q=0), -1),
    ({}, dict(rows=0, weight=0, pool=0, slot_map=0, rows_out=0, q=0, q_weight=0, q_out=0), -1),
    (dict(pool_format=m.MLA_POOL_NONE), dict(pool=0, slot_map=0, rows_out=0), -1), (dict(pool_format=m.MLA_POOL_NONE), {}, -1),
    (dict(row_stride=584), dict(rows=3 * X, rows_out=3 * X), -1), (dict(q_token_stride=8 * 200), dict(q=X, q_out=X), -1),
    (dict(q_head_stride=200), dict(q=X, q_out=X), -1), (dict(num_rows=0), {}, 0),
])
def test_rope_append_refuses(lib, desc, args, want):
    a = dict(rows=X, weight=X, q=X, q_weight=X, positions=X, cos_sin=X, slot_map=X, pool=X, rows_out=2 * X, q_out=2 * X, debug=0)
    a.update(args)
    p = [a[k] or None for k in ("rows", "weight", "q", "q_weight", "positions", "cos_sin", "slot_map", "pool", "rows_out", "q_out")]
    assert lib.mla_rope_append(ctypes.byref(rope_desc(**desc)), *p, a["debug"], None, None) == want


def test_wrappers_refuse_tensors_on_the_host():
    import torch
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.rope_append(None, torch.zeros(4, 576, dtype=torch.bfloat16), None, i32, torch.zeros(8, 64))
    q = torch.zeros(4, 2, 192, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.prompt_attn(q, q[..., :128], q[:, 0, 128:], q[..., :128], i32[:2], max_q_len=4)
