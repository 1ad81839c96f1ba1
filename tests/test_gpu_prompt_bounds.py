"""The bounds that a caller of mla_prompt_attn names (include/mla_prompt.h), and what is made of them where they are left out."""
import numpy as np
import pytest

from _helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()


def ints(v):
    return to_dev(np.asarray(v, np.int32))


def problem(nq, nk, heads=2, seed=1):
    import torch
    rng = np.random.default_rng(seed)
    normal = lambda *shape: torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(torch.bfloat16).cuda()
    return dict(q=normal(nq, heads, 192), k_nope=normal(nk, heads, 128), k_rope=normal(nk, 64), v=normal(nk, heads, 128))


@pytest.mark.parametrize("m,n", [([17], [900]), ([1, 1, 1], [300, 5, 140]), ([40, 3], [40, 3]), ([9, 4], [3, 0])])
def test_keys_of_their_own_are_all_read_without_a_bound(m, n):
    """cu_k given and max_k_len not: as with the bound named, whatever the queries' bound is."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p = problem(sum(m), sum(n))
    cu_q, cu_k = (ints(np.concatenate([[0], np.cumsum(v)])) for v in (m, n))
    out, lse = lib.prompt_attn(**p, cu_q=cu_q, cu_k=cu_k, max_q_len=max(m))
    want = lib.prompt_attn(**p, cu_q=cu_q, cu_k=cu_k, max_q_len=max(m), max_k_len=sum(n))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    plain = lib.prompt_attn(**p, cu_q=cu_q, cu_k=cu_k, max_q_len=max(m), max_k_len=sum(n), flags=lib.MLA_FLAG_SIMT)
    seen = torch.isfinite(plain[1])
    assert torch.equal(seen, torch.isfinite(lse)) and torch.allclose(lse[seen], plain[1][seen], atol=2e-4)


def test_without_keys_of_their_own_the_queries_bound_holds():
    import torch
    import speculative_decode_mla_gb300 as lib
    p = problem(70, 70)
    out, lse = lib.prompt_attn(**p, cu_q=ints([0, 30, 70]), max_q_len=40)
    want = lib.prompt_attn(**p, cu_q=ints([0, 30, 70]), cu_k=ints([0, 30, 70]), max_q_len=40, max_k_len=40)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("log2_scale", [127, 100, 0, -100, -149])
def test_scales_to_the_ends_of_their_range(log2_scale, flags):
    """Queries that undo the scale as far as bf16 goes: scores as float64 has them (powers of two leave every other rounding as it is)."""
    import oracle
    import speculative_decode_mla_gb300 as lib
    p = problem(150, 400, heads=1, seed=3)
    p["q"].mul_(2.0 ** max(-60, min(90, -log2_scale // 2)))
    for k in ("k_nope", "k_rope"):
        p[k].mul_(2.0 ** max(-60, min(30, -log2_scale - (-log2_scale // 2) - 3)))
    scale = 2.0 ** log2_scale
    out, lse = lib.prompt_attn(**p, cu_q=ints([0, 150]), cu_k=ints([0, 400]), max_q_len=150, max_k_len=400, softmax_scale=scale,
                               flags=lib.MLA_FLAG_SIMT if flags == "simt" else 0)
    host = lambda t: t.double().cpu().numpy()
    o, l, spread, size = oracle.prompt_attn(*(host(p[k]) for k in ("q", "k_nope", "k_rope", "v")), [0, 150], [0, 400], causal=True, scale=scale)
    e = 256 * 2.0 ** -23 * size      # the tolerances of test_gpu_prompt.py
    assert (np.abs(host(lse) - l) <= e + 2.0 ** -20 * (1 + np.abs(l))).all()
    assert (np.abs(host(out) - o) <= (2.0 ** -8 + 2.5 * e + 2.0 ** -19)[..., None] * spread + 2.0 ** -8 * np.abs(o) + 1e-30).all()


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("cu_q,cu_k,rows,most_q,bad", [
    ([0, 5], [0, 9], 5, 0, True),                # no room for a query, and five of them
    ([0, 5], [0, 9], 0, 5, True),                # no rows at all
    ([0, 5, 5], [0, 9, 30], 5, 5, True),         # a sequence without queries whose keys end outside
    ([5, 0, 5], [0, 9, 9], 5, 5, True),          # ends that fall
    ([0, 5, 5], [0, 9, 9], 5, 5, False), ([0, 0], [0, 0], 0, 0, False), ([2, 2, 2], [1, 1, 9], 5, 5, False),
])
def test_debug_checks_see_sequences_that_no_row_belongs_to(cu_q, cu_k, rows, most_q, bad, flags):
    import torch
    import speculative_decode_mla_gb300 as lib
    p = problem(5, 9)
    p["q"] = p["q"][:rows]
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    call = lambda: lib.prompt_attn(**p, cu_q=ints(cu_q), cu_k=ints(cu_k), max_q_len=most_q, max_k_len=9, dev_status=status,
                                   flags=lib.MLA_FLAG_DEBUG_CHECKS | (lib.MLA_FLAG_SIMT if flags == "simt" else 0))
    if bad:
        with pytest.raises(lib.MLAError):
            call()
    else:
        call()
    assert int(status) == (lib.CHECK_BAD_LENGTH if bad else 0)


@pytest.mark.parametrize("bound", [2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 63 - 1])
def test_bounds_past_32_bits(bound):
    """An upper bound may be any number; no sequence has more rows than its tensor."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p = dict(problem(60, 300), cu_q=ints([0, 40, 60]), cu_k=ints([0, 200, 300]))
    want = lib.prompt_attn(**p, max_q_len=60, max_k_len=300)
    got = lib.prompt_attn(**p, max_q_len=bound, max_k_len=bound)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(lib.MLAError):
        lib.prompt_attn(**p, max_q_len=-1, max_k_len=bound)
    with pytest.raises(lib.MLAError):
        lib.prompt_attn(**p, max_q_len=bound, max_k_len=-2 ** 32 + 300)
