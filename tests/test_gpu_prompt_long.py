"""mla_prompt_attn over many keys (include/mla_prompt.h): sums that do not lose as they grow.

Tolerances are those of test_gpu_prompt.py, which do not grow with the number of keys: e = 256 * 2^-23 of sum |q||k| times the scale for
the scores, |lse error| <= e + 2^-20 (1 + |lse|), |out error| <= (2^-8 + 2.5 e + 2^-19) * sum of weights |values| + 2^-8 |out|.
The sum of 2^17 weights of about 1, taken one by one in float32, is off by 2^-12 and more: each addend is rounded to the last place of a
total up to 2^17 times its size, equal ones always the same way.
"""
import numpy as np
import pytest

import oracle
from _helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()


def inputs(m, n, scores, seed=1):
    """m equal queries and n keys of one head; key t's score is scores[t] (rounded to bf16), from the keys' own dims or the RoPE dims."""
    import torch
    b = dict(dtype=torch.bfloat16, device="cuda")
    q, k, kr = torch.zeros(m, 1, 192, **b), torch.zeros(n, 1, 128, **b), torch.zeros(n, 64, **b)
    v = to_dev(np.random.default_rng(seed).normal(size=(n, 1, 128)).astype(np.float32)).to(torch.bfloat16)
    q[..., 5], q[..., 131] = 1.0, 1.0
    s = to_dev(scores.astype(np.float32)).to(torch.bfloat16)
    k[::2, 0, 5], kr[1::2, 3] = s[::2], s[1::2]
    return q, k, kr, v


def scores_of(kind, n):
    s = np.full(n, -0.0203) if kind == "equal" else np.random.default_rng(3).uniform(-0.5, -0.01, n)
    s[0] = 0.0       # the largest, in the first tile: all later weights are added to its sum
    return s


@pytest.mark.parametrize("kind", ["equal", "spread"])
@pytest.mark.parametrize("m,n,how", [(1, 131072 + 37, "one cta"), (200, 70001, "one cta"), (1, 131072 + 37, "shared"), (200, 70001, "shared"),
                                     (608 * 256, 66000, "units"), (3, 70001, "simt")])
def test_sums_over_many_keys(m, n, how, kind):
    import torch
    import speculative_decode_mla_gb300 as lib
    q, k, kr, v = inputs(m, n, scores_of(kind, n))
    ends = lambda e: to_dev(np.array([0, e], np.int32))
    out, lse = lib.prompt_attn(q, k, kr, v, ends(m), ends(n), max_q_len=m, max_k_len=n, causal=False, softmax_scale=1.0,
                               num_ctas=1 if how == "one cta" else 0, out_dtype=lib.MLA_DTYPE_F32, flags=lib.MLA_FLAG_SIMT if how == "simt" else 0)
    assert (out == out[:1]).all() and (lse == lse[0]).all() or how == "shared"     # equal queries (parts may end inside a row tile)
    host = lambda t: t.double().cpu().numpy()
    o, l, spread, size = oracle.prompt_attn(host(q[:1]), host(k), host(kr), host(v), [0, 1], [0, n], causal=False, scale=1.0)
    e = 256 * 2.0 ** -23 * size[0, 0]
    off = (lse.double() - float(l[0, 0])).abs().max().item()
    assert off <= e + 2.0 ** -20 * (1 + abs(l[0, 0])), off
    off = np.abs(host(out[:256]) - o) - (2.0 ** -8 + 2.5 * e + 2.0 ** -19) * spread
    assert off.max() <= 0, off.max()
