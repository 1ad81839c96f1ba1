"""mla_prompt_attn in calls of many units (include/mla_prompt.h): whole units of two lanes that CTAs claim one after the other, listed longest
first, heads in groups. Every plan is looked at first, so that a call runs the way that it is here for. Tolerances are those of test_gpu_prompt.py.
"""
import numpy as np
import pytest

import oracle
from test_gpu_prompt import SCALE, Problem, check, ends, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()
    oracle.build()


def plan(p, most_k=None, **kw):
    """The plan of p.run()."""
    import torch
    import speculative_decode_mla_gb300 as lib
    d = lib.PromptDesc(num_seqs=len(p.m), num_heads=p.heads, num_kv_heads=p.k.shape[1], max_q_len=max(p.m), max_k_len=most_k or max(p.n), causal=1,
                       softmax_scale=SCALE, num_q=p.q.shape[0], num_k=p.k.shape[0], q_token_stride=p.q.stride(0), q_head_stride=p.q.stride(1),
                       k_token_stride=p.k.stride(0), k_head_stride=p.k.stride(1), k_rope_token_stride=p.kr.stride(0), v_token_stride=p.v.stride(0),
                       v_head_stride=p.v.stride(1), **kw)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return lib.prompt_plan(d, sms), sms


def head_groups(p, pack):
    """(virtual heads, of a group) of a call: 48 MB of keys and values a group (kGroupBytes)."""
    virtual, group = p.heads // pack, p.heads // p.k.shape[1]
    return virtual, min(virtual, max(1, (48 << 20) // (p.k.shape[0] * 512)) * (group // pack))


def exact(p, causal=True):
    """oracle.prompt_attn's four results for a problem, in float64 on the device: it takes large ones too."""
    import torch
    out = torch.full((p.q.shape[0], p.heads, 128), float("nan"), dtype=torch.float64, device="cuda")
    spread, lse, size = out.clone(), out[:, :, 0].clone(), out[:, :, 0].clone()
    for b in range(len(p.m)):
        m, n, q0, k0 = p.m[b], p.n[b], int(p.cu_q[b]), int(p.cu_k[b])
        for g in range(p.k.shape[1]):
            heads = slice(g * (p.heads // p.k.shape[1]), (g + 1) * (p.heads // p.k.shape[1]))
            key = torch.cat([p.k[k0:k0 + n, g], p.kr[k0:k0 + n]], 1).double()
            val, q = p.v[k0:k0 + n, g].double(), p.q[q0:q0 + m, heads].double()
            s, mag = q @ key.T * SCALE, q.abs() @ key.abs().T * SCALE
            if causal:
                hidden = torch.arange(n, device="cuda") > torch.arange(m, device="cuda")[:, None] + n - m
                s.masked_fill_(hidden[:, None], -float("inf"))
                mag.masked_fill_(hidden[:, None], 0.0)
            l = torch.logsumexp(s, 2) if n else torch.full(s.shape[:2], -float("inf"), dtype=torch.float64, device="cuda")
            w = torch.exp(s - torch.where(torch.isfinite(l), l, 0.0)[..., None])
            rows = slice(q0, q0 + m)
            out[rows, heads], spread[rows, heads], lse[rows, heads] = w @ val, w @ val.abs(), l
            size[rows, heads] = mag.amax(2) if n else 0.0
    return tuple(t.cpu().numpy() for t in (out, lse, spread, size))


def same(a, b):
    import torch
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("causal", [True, False])
def test_the_device_reference_is_the_oracle(causal):
    p = Problem([5, 0, 30, 4], [9, 3, 30, 0], 4, 2, seed=2)
    for a, b in zip(exact(p, causal), p.want(causal)):
        assert np.allclose(a, b, equal_nan=True, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("heads,group", [(8, 1), (12, 2), (9, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_units_that_are_claimed(causal, heads, group):
    """Several units of two lanes a CTA: of one row tile and of two, with and without a second lane, of 1 to 500 rows and keys."""
    rng = np.random.default_rng(heads)
    m = [int(v) for v in rng.integers(1, 501, 60)]
    m[3] = m[17] = m[59] = 0
    m[5], m[6] = 500, 1
    n = [min(512, v + int(e)) for v, e in zip(m, rng.choice([0, 0, 7, 200], 60))]
    n[8] = 3                                     # fewer keys than queries
    p = Problem(m, n, heads, group, seed=heads)
    what, sms = plan(p)
    assert not what.shared and what.listed and what.rows_per_unit == 256 and what.ctas > 2 * sms
    got = p.run(causal=causal)
    check(got, exact(p, causal))
    for _ in range(3):
        assert same(p.run(causal=causal), got)


@pytest.mark.parametrize("m,n,heads,group", [([2100], [2100], 80, 1), ([2100], [2100], 160, 2), ([1500], [2200], 180, 3),
                                             ([2500, 129, 0, 700, 1800, 256, 1, 1025, 40, 333, 2111, 900], [2500, 400, 9, 700, 3000, 256, 1, 1025, 40, 340, 2111, 900], 25, 1),
                                             ([2000, 60, 900, 1300], [2000, 2500, 900, 1400], 96, 4)])
def test_heads_in_groups(m, n, heads, group):
    """Units of many tiles, in more than one group of heads, the last of them smaller; of one sequence, and listed."""
    p = Problem(m, n, heads, group, seed=len(m) + heads)
    what, sms = plan(p)
    assert not what.shared and what.listed == (len(m) > 1) and what.rows_per_unit == 256 and what.ctas > 2 * sms
    virtual, of_group = head_groups(p, what.pack)
    assert of_group < virtual and virtual % of_group != 0
    got = p.run()
    check(got, exact(p))
    assert same(p.run(), got)


def test_keys_that_need_a_coarser_list():
    """More key tiles than the list's sort has bins: one sequence of 270,000 keys among 619 short ones."""
    rng = np.random.default_rng(5)
    m = [int(v) for v in rng.integers(0, 41, 620)]
    m[11], m[12] = 40, 40
    n = [v + int(e) for v, e in zip(m, rng.choice([0, 5, 300], 620))]
    n[11] = 270000
    p = Problem(m, n, 8, 8, seed=5)
    what, sms = plan(p)
    assert not what.shared and what.listed and what.rows_per_unit == 256 and max(n) / 128 >= 2048
    got = p.run()
    check(got, exact(p))
    assert same(p.run(), got)


@pytest.mark.parametrize("m,n,heads", [([300, 1, 500, 64, 129, 31, 256, 411, 2] * 3, None, 24), ([300, 290, 400], [1500, 300, 700], 304)])
def test_a_sequence_alone_and_among_others(m, n, heads):
    """The same bits in every order that units are claimed in: in the batch, several times over, and alone."""
    import speculative_decode_mla_gb300 as lib
    p = Problem(m, n or m, heads, seed=heads)
    what, sms = plan(p)
    assert not what.shared and what.listed and what.rows_per_unit == 256 and what.ctas > 2 * sms
    got = p.run()
    for _ in range(5):
        assert same(p.run(), got)
    for i in range(min(9, len(m))):
        (q0, q1), (k0, k1) = p.cu_q[i:i + 2], p.cu_k[i:i + 2]
        alone = Problem.__new__(Problem)
        alone.m, alone.n, alone.heads, alone.cu_q, alone.cu_k = [m[i]], [int(k1 - k0)], heads, ends([m[i]]), ends([int(k1 - k0)])
        alone.q, alone.k, alone.kr, alone.v = p.q[q0:q1], p.k[k0:k1], p.kr[k0:k1], p.v[k0:k1]
        assert not plan(alone)[0].shared
        assert same(alone.run(), (got[0][q0:q1], got[1][q0:q1])), i


def test_one_cta_and_whole_units():
    """Named CTAs make a shared call: with one of them every unit is whole, in the sequences' order, and the bits are those of claimed units."""
    import speculative_decode_mla_gb300 as lib
    m = [300, 1, 500, 64, 129, 31, 256, 411, 2] * 2
    p = Problem(m, m, 20, seed=7)
    assert not plan(p)[0].shared and plan(p, num_ctas=1)[0].shared
    assert same(p.run(), p.run(num_ctas=1))
