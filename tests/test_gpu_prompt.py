"""GPU parity of mla_prompt_attn (include/mla_prompt.h) with the float64 oracle, and of the prompt's steps together.

Tolerance, per element. Scores: 192 exact products added in float32, off by at most e = 256 * 2^-23 of sum |q||k| (times the scale); a
weight, after its division by the sum, by a factor of 1 +- 2.5 e, and 2^-20 for exp2, sums and parts. A weight is rounded to
bf16 (2^-8 at most of itself) and so, with a bf16 output, is the result (2^-8 of itself); so
|out error| <= (2^-8 + 2.5 e + 2^-19) * sum of weights |values| + 2^-8 |out|, and |lse error| <= e + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

import oracle
from _helpers import to_dev

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()
    oracle.build()


def values(t):
    return t.double().cpu().numpy()


def normal(rng, *shape, scale=1.0):
    import torch
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def ints(v):
    return to_dev(np.asarray(v, np.int32))


def ends(lengths, start=0):
    return np.concatenate([[start], start + np.cumsum(lengths)]).astype(np.int32)


class Problem:
    """Packed sequences with m[b] queries and n[b] keys; `before`, `behind`: rows outside the sequences."""

    def __init__(self, m, n, heads, group=1, seed=1, scale=1.0, before=0, behind=0):
        rng = np.random.default_rng(seed)
        self.cu_q, self.cu_k, self.m, self.n, self.heads, hk = ends(m, before), ends(n, before), m, n, heads, heads // group
        nq, nk = int(self.cu_q[-1]) + behind, int(self.cu_k[-1]) + behind
        self.q = normal(rng, nq, heads, 192, scale=scale)
        kv = normal(rng, nk, hk, 256)
        self.kv, self.k, self.v = kv, kv[..., :128], kv[..., 128:]
        self.rows = normal(rng, nk, 576)
        self.kr = self.rows[:, 512:]

    def want(self, causal=True, scale=SCALE):
        return oracle.prompt_attn(values(self.q), values(self.k), values(self.kr), values(self.v), self.cu_q, self.cu_k, causal=causal, scale=scale)

    def run(self, **kw):
        import speculative_decode_mla_gb300 as m
        kw.setdefault("max_q_len", max(self.m))
        kw.setdefault("max_k_len", max(self.n))
        return m.prompt_attn(self.q, self.k, self.kr, self.v, ints(self.cu_q), ints(self.cu_k), **kw)


def check(got, want, f32=False):
    out, lse = values(got[0]), values(got[1])
    o, l, spread, size = want
    real = ~np.isnan(l)
    o, spread, out = o[real], spread[real], out[real]
    l, size, lse = l[real], size[real], lse[real]
    e = 256 * 2.0 ** -23 * size
    off = np.abs(out - o) - ((2.0 ** -8 + 2.5 * e + 2.0 ** -19)[:, None] * spread + (0.0 if f32 else 2.0 ** -8) * np.abs(o) + 1e-30)
    assert off.max() <= 0, ("out", off.max(), np.abs(out - o).max())
    none = np.isneginf(l)
    assert (np.isneginf(lse) == none).all()
    off = np.abs(lse[~none] - l[~none]) - (e[~none] + 2.0 ** -20 * (1 + np.abs(l[~none])))
    assert off.size == 0 or off.max() <= 0, ("lse", off.max())


CASES = [
    # (queries, keys, heads, group)
    ([1], [1], 1, 1), ([2], [2], 3, 1), ([61], [61], 8, 1), ([127], [127], 2, 1), ([128], [128], 2, 1), ([129], [129], 2, 1),
    ([255], [255], 1, 1), ([256], [256], 2, 2), ([257], [257], 1, 1), ([513], [513], 2, 1), ([1000], [1000], 2, 1),
    ([1], [1000], 4, 4), ([1], [128], 2, 1), ([17], [2049], 4, 2), ([130], [700], 3, 3), ([300], [301], 2, 1), ([256], [640], 1, 1),
    ([5, 200, 1, 64, 129, 0, 33], [5, 200, 1, 64, 129, 0, 33], 4, 2), ([3, 0, 70, 1], [400, 9, 71, 1], 4, 1),
    ([1] * 9, [1, 2, 127, 128, 129, 255, 256, 257, 600], 4, 4), ([5, 300, 10], [2, 100, 0], 2, 1), ([200, 4], [0, 7], 2, 1),
]


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("m,n,heads,group", CASES)
def test_against_the_oracle(m, n, heads, group, causal, flags):
    import speculative_decode_mla_gb300 as lib
    p = Problem(m, n, heads, group, seed=sum(m) + heads)
    check(p.run(causal=causal, flags=lib.MLA_FLAG_SIMT if flags == "simt" else 0), p.want(causal))


@pytest.mark.parametrize("m,n,heads,group", [([70, 300, 1, 0, 40], [900, 300, 515, 3, 2], 2, 2), ([700], [2500], 3, 1),
                                             ([5, 60, 1, 2], [1300, 64, 2000, 700], 2, 1), ([2000], [2000], 2, 1), ([90, 40], [1000, 3], 8, 8)])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40, 500])
def test_shared_by_any_number_of_ctas(ctas, m, n, heads, group):
    import speculative_decode_mla_gb300 as lib
    p = Problem(m, n, heads, group, seed=4)
    for causal in (True, False):
        check(p.run(num_ctas=ctas, causal=causal), p.want(causal))
    check(p.run(num_ctas=ctas, out_dtype=lib.MLA_DTYPE_F32), p.want(), f32=True)


@pytest.mark.parametrize("heads,group", [(6, 3), (8, 8), (32, 32), (128, 128), (10, 5), (16, 4)])
def test_grouped_heads(heads, group):
    p = Problem([3, 70, 1], [50, 200, 140], heads, group, seed=heads)
    for ctas in (0, 5):
        for causal in (True, False):
            check(p.run(num_ctas=ctas, causal=causal), p.want(causal))


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("ctas", [0, 1, 3])
def test_rows_outside_the_sequences_are_left_alone(ctas, flags):
    """Rows before the first and behind the last sequence: not written, and NaN and infinities there reach nothing."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p = Problem([40, 130], [90, 200], 2, seed=5, before=3, behind=140)
    clean = p.want()
    for t, lo, hi in ((p.q, 3, 173), (p.kv, 3, 293), (p.rows, 3, 293)):
        t[:lo], t[hi:] = float("nan"), float("inf")
    out = torch.full((p.q.shape[0], 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.q.shape[0], 2), 7.0, device="cuda")
    got = p.run(out=out, lse=lse, num_ctas=ctas, flags=lib.MLA_FLAG_SIMT if flags == "simt" else 0)
    assert got[0] is out and got[1] is lse
    check(got, clean)
    for t in (out, lse):
        assert (t[:3] == 7).all() and (t[173:] == 7).all()


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("what", ["k", "kr", "v"])
@pytest.mark.parametrize("m,n,at", [([300], [300], [(0, 150)]), ([300], [300], [(0, 0)]), ([300], [400], [(0, 399), (0, 300), (0, 130)]),
                                    ([129], [129], [(0, 128)]), ([100, 60, 200], [100, 60, 200], [(1, 0), (1, 59), (0, 99), (2, 127)]),
                                    ([64], [512], [(0, 460)])])
def test_what_a_row_does_not_see_does_not_reach_it(m, n, at, what, ctas):
    """NaN and infinities in keys and values: rows that see them are not finite where they are not, all others as without them."""
    import torch
    p = Problem(m, n, 2, seed=6)
    good = p.run(num_ctas=ctas)
    odd = [float("nan"), float("inf"), float("-inf")]
    for i, (b, t) in enumerate(at):
        row = int(p.cu_k[b]) + t
        if what == "v":
            p.kv[row, i % 2, 128 + 5 * i] = odd[i % 3]
            p.kv[row, i % 2, 128 + 5 * i + 64] = odd[(i + 1) % 3]
        elif what == "k":
            p.kv[row, i % 2, 7 * i] = float("nan")
        else:
            p.rows[row, 512 + i] = float("nan")
    got = p.run(num_ctas=ctas)
    out, want = values(got[0]), values(good[0])
    touched = np.zeros(out.shape, bool)
    for i, (b, t) in enumerate(at):
        for j in range(m[b]):
            if t <= j + n[b] - m[b]:
                r = int(p.cu_q[b]) + j
                if what == "v":
                    touched[r, i % 2, [5 * i, 5 * i + 64]] = True
                else:
                    touched[r, i % 2 if what == "k" else slice(None)] = True
    assert np.isfinite(out[~touched]).all() and not np.isfinite(out[touched]).any()
    assert np.array_equal(out[~touched], want[~touched])
    if what == "v":
        assert torch.equal(got[1], good[1])
        o, _, _, _ = p.want()
        assert np.array_equal(np.isnan(out), np.isnan(o)) and np.array_equal(out[np.isinf(out)], o[np.isinf(out)])


@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("scale", [8.0, 3e4, 1e9])
def test_large_scores(scale, ctas):
    """Queries so large that the softmax picks one key: out is its value, or a mean of keys whose scores are equal in float32."""
    p = Problem([150], [420], 2, seed=7, scale=scale)
    out, lse = (values(t) for t in p.run(num_ctas=ctas))
    o, l, _, size = p.want()
    ok = np.abs(out - o).max(-1) <= 0.02
    q, k = values(p.q), np.concatenate([values(p.k), np.repeat(values(p.kr)[:, None], 2, 1)], 2)
    s = np.einsum("ihd,thd->iht", q, k) * SCALE
    for i in range(150):
        s[i, :, i + 271:] = -np.inf
    two = np.sort(s, 2)[..., -2:]
    clear = two[..., 1] - two[..., 0] > 2 * 256 * 2.0 ** -23 * size + 8        # the largest stands apart by more than rounding
    assert clear.mean() > 0.05 or scale == 8.0
    assert (ok | ~clear).all() and np.isfinite(out).all()
    assert (np.abs(lse - l) <= 256 * 2.0 ** -23 * size + 2.0 ** -20 * (1 + np.abs(l))).all()


def test_growing_maxima():
    """Scores that rise along the keys (each tile's maximum well above the last): the output is rescaled at every tile."""
    import torch
    p = Problem([260], [1500], 2, seed=8)
    t = torch.arange(1500, device="cuda").float()
    p.kv[:, :, :128] *= (0.2 + t / 300)[:, None, None].to(torch.bfloat16)
    check(p.run(num_ctas=1), p.want())
    check(p.run(num_ctas=4), p.want())


@pytest.mark.parametrize("layout", ["heads_first", "wide", "one"])
def test_strides(layout):
    import torch
    import speculative_decode_mla_gb300 as lib
    p = Problem([90, 150], [120, 150], 4, 2, seed=9)
    want = lib.prompt_attn(p.q, p.k.contiguous(), p.kr.contiguous(), p.v.contiguous(), ints(p.cu_q), ints(p.cu_k), max_q_len=150, max_k_len=150)
    if layout == "heads_first":
        first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
        q, k, kr, v = first(p.q), first(p.k), p.kr, first(p.v)
    elif layout == "wide":
        pad = lambda t, by: torch.nn.functional.pad(t, by)[..., by[0]:by[0] + t.shape[-1]]
        q, k, kr, v = pad(p.q, (8, 16)), pad(p.k, (0, 24)), pad(p.kr, (64, 8)), pad(p.v, (40, 0))
    else:
        q, k, kr, v = p.q[:, 1:2], p.k[:, :1], p.kr, p.v[:, :1]
        want = want[0][:, 1:2].contiguous(), want[1][:, 1:2].contiguous()
    got = lib.prompt_attn(q, k, kr, v, ints(p.cu_q), ints(p.cu_k), max_q_len=150, max_k_len=150)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_results_do_not_depend_on_the_batch():
    """A sequence alone and among others: the same bits (with whole units), whatever order the units run in; and twice the same bits."""
    import torch
    m = [300, 1, 700, 64, 129, 31, 256, 999, 2]
    p = Problem(m, m, 3, seed=10)
    a, b = p.run(num_ctas=1), p.run(num_ctas=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    import speculative_decode_mla_gb300 as lib
    for i in range(len(m)):
        lo, hi = int(p.cu_q[i]), int(p.cu_q[i + 1])
        out, lse = lib.prompt_attn(p.q[lo:hi], p.k[lo:hi], p.kr[lo:hi], p.v[lo:hi], ints([0, m[i]]), max_q_len=m[i], num_ctas=1)
        assert torch.equal(out, a[0][lo:hi]) and torch.equal(lse, a[1][lo:hi])


@pytest.mark.parametrize("seqs,most", [(3000, 3), (40, 400)])
def test_many_sequences(seqs, most):
    import torch
    import speculative_decode_mla_gb300 as lib
    rng = np.random.default_rng(seqs)
    m = rng.integers(0, most + 1, seqs)
    n = m + rng.integers(0, 2 * most, seqs)
    p = Problem(m.tolist(), n.tolist(), 2, seed=11)
    a, b = p.run(), p.run(flags=lib.MLA_FLAG_SIMT)
    assert torch.allclose(a[0].float(), b[0].float(), atol=0.03, rtol=0.02)
    fine = torch.isfinite(b[1])
    assert torch.equal(fine, torch.isfinite(a[1])) and torch.allclose(a[1][fine], b[1][fine], atol=2e-4)
    if most > 100:
        check(a, p.want())


@pytest.mark.parametrize("ctas", [1, 37, 152, 1000])
@pytest.mark.parametrize("most", [1500, 60])
def test_shares_of_a_large_batch(ctas, most):
    """Shares that begin in any of a hundred sequences, empty ones and ones of many row tiles among them, with one and two lanes."""
    rng = np.random.default_rng(most)
    m = [int(v) for v in np.minimum(most, rng.choice([0, 1, 3, 60, 130, 700, 1500], 100, p=[.2, .3, .2, .2, .06, .02, .02]))]
    m[0], m[31], m[32], m[-1] = 0, most, 0, most
    n = [v + int(e) for v, e in zip(m, rng.choice([0, 5, 200], 100))]
    p = Problem(m, n, 2, seed=21)
    check(p.run(num_ctas=ctas), p.want())


def test_lengths_are_read_on_the_device():
    """A call with room for more, captured, then replayed with other lengths and data: as an eager call with those."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p = Problem([200, 90, 160], [260, 90, 400], 2, seed=12)
    cu_q, cu_k = ints(p.cu_q), ints(p.cu_k)
    desc_out, lse = torch.zeros(450, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(450, 2, device="cuda")
    call = lambda **kw: lib.prompt_attn(p.q, p.k, p.kr, p.v, cu_q, cu_k, max_q_len=300, max_k_len=500, **kw)
    for ctas in (0, 1, 3):
        call(num_ctas=ctas)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(num_ctas=ctas, out=desc_out, lse=lse)
        for m, n in (([200, 90, 160], [260, 90, 400]), ([1, 300, 2], [1, 310, 400]), ([0, 0, 5], [200, 50, 500])):
            cu_q.copy_(ints(ends(m)))
            cu_k.copy_(ints(ends(n)))
            p.q.copy_(normal(np.random.default_rng(sum(m)), *p.q.shape))
            desc_out.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            p.cu_q, p.cu_k = ends(m), ends(n)
            check((desc_out, lse), p.want())
            assert (desc_out[sum(m):] == 7).all()


@pytest.mark.parametrize("m,heads", [(1, 4), (100, 1), (200, 1)])
def test_repeated_with_cold_caches(m, heads):
    """Some tiles a unit, with the caches swept before every call, so that loads are late: always the same bits."""
    import torch
    p = [Problem([m], [n], heads, heads, seed=n) for n in (300, 384, 640, 1000, 1400)] + [Problem([m] * 5, [200, 384, 900, 129, 700], heads, heads, seed=2)]
    sweep = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = {}
    for i in range(24):
        for k, x in enumerate(p):
            for causal in (True, False):
                sweep.fill_(i)
                got = x.run(num_ctas=i % 3, causal=causal)
                was = first.setdefault((k, i % 3, causal), got)
                assert torch.equal(got[0], was[0]) and torch.equal(got[1], was[1]), (i, k, causal)
                if i < 3:
                    check(got, x.want(causal))


def test_two_streams_at_once():
    import torch
    a, b = Problem([700, 30], [700, 900], 2, seed=13), Problem([40] * 12, [333] * 12, 4, seed=14)
    want = [p.run() for p in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got = [p.run(stream=s) for p, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_debug_checks_report_bad_ends():
    import torch
    import speculative_decode_mla_gb300 as lib
    p = Problem([50, 60], [50, 60], 2, seed=15)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=lib.MLA_FLAG_DEBUG_CHECKS, dev_status=status)
    p.run(**kw)
    assert int(status) == 0
    for cu_q, cu_k, most in (([0, 50, 111], [0, 50, 110], 60), ([0, 50, 110], [0, 50, 200], 60), ([0, 60, 50], [0, 50, 110], 60), ([-1, 50, 110], [0, 50, 110], 60),
                             ([0, 50, 110], [0, 50, 110], 59)):
        with pytest.raises(lib.MLAError):
            lib.prompt_attn(p.q, p.k, p.kr, p.v, ints(cu_q), ints(cu_k), max_q_len=most, max_k_len=60, **kw)
        assert int(status) == lib.CHECK_BAD_LENGTH
        lib.prompt_attn(p.q, p.k, p.kr, p.v, ints(cu_q), ints(cu_k), max_q_len=most, max_k_len=60)  # clamped, no fault
        lib.prompt_attn(p.q, p.k, p.kr, p.v, ints(cu_q), ints(cu_k), max_q_len=most, max_k_len=60, num_ctas=2)
    torch.cuda.synchronize()


def test_nothing_to_do():
    import torch
    import speculative_decode_mla_gb300 as lib
    b = dict(dtype=torch.bfloat16, device="cuda")
    q, k, kr = torch.zeros(0, 4, 192, **b), torch.zeros(5, 2, 128, **b), torch.zeros(5, 64, **b)
    out, lse = lib.prompt_attn(q, k, kr, k, ints([0, 0]), ints([0, 5]), max_q_len=3, max_k_len=5)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    q = torch.ones(7, 4, 192, **b)
    for causal in (True, False):
        out, lse = lib.prompt_attn(q, k[:0], kr[:0], k[:0], ints([0, 7]), ints([0, 0]), max_q_len=7, max_k_len=0, causal=causal)
        assert (out == 0).all() and torch.isneginf(lse).all()


def test_wrapper_refuses():
    import torch
    import speculative_decode_mla_gb300 as lib
    p = Problem([5], [5], 4, 2, seed=16)
    good = dict(q=p.q, k_nope=p.k, k_rope=p.kr, v=p.v, cu_q=ints([0, 5]), cu_k=ints([0, 5]), max_q_len=5)
    lib.prompt_attn(**good)
    for bad in (dict(q=p.q.float()), dict(q=p.q[..., :128]), dict(k_nope=p.kv), dict(k_rope=p.rows), dict(k_rope=p.kr[:4]), dict(v=p.v[:4]),
                dict(v=p.v[:, :1]), dict(cu_q=ints([0, 5]).long()), dict(cu_k=ints([0, 2, 5])), dict(q=p.q.cpu()), dict(k_nope=p.kv[..., ::2]),
                dict(out=torch.zeros(5, 4, 128, device="cuda")), dict(lse=torch.zeros(4, 5, device="cuda")), dict(k_nope=p.k.half())):
        with pytest.raises(ValueError):
            lib.prompt_attn(**{**good, **bad})
    for bad in (dict(k_nope=p.k[:, :1].expand(-1, 3, -1), v=p.v[:, :1].expand(-1, 3, -1)), dict(max_q_len=-1), dict(num_ctas=2000), dict(softmax_scale=0.0),
                dict(q=p.q[:, :1].expand(-1, 4, -1)), dict(flags=64), dict(k_rope=torch.zeros(5, 65, dtype=torch.bfloat16, device="cuda")[:, 1:])):
        with pytest.raises(lib.MLAError):
            lib.prompt_attn(**{**good, **bad})


@pytest.mark.parametrize("fmt", ["bf16", "kv4"])
def test_prompt_then_decode(fmt):
    """A layer as a server runs it. The prompt: norms, rotations, rows into the pool, expansion, prompt attention, once whole and once in
    two chunks. Then the last token again as a decode step: its absorbed query against the pool; both ways give one attention."""
    import torch
    import speculative_decode_mla_gb300 as lib
    rng = np.random.default_rng(17)
    n, heads = 333, 4
    rows, q = normal(rng, n, 576), normal(rng, n, heads, 192)
    w, qw = normal(rng, 512), normal(rng, 192)
    a = np.arange(2000)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    table = to_dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
    pos, slots = to_dev(np.arange(n, dtype=np.int32) + 100), to_dev(rng.permutation(500)[:n].astype(np.int32))
    pool = torch.zeros(500, 576, dtype=torch.bfloat16, device="cuda") if fmt == "bf16" else torch.zeros(500, 416, dtype=torch.uint8, device="cuda")
    rows_out, q_out = lib.rope_append(pool, rows, slots, pos, table, weight=w, q=q, q_weight=qw)
    held = rows_out if fmt == "bf16" else lib.kv4_gather(pool, slots)      # what the pool stands for
    wk, wv = normal(rng, heads, 512, 128, scale=512 ** -0.5), normal(rng, heads, 512, 128, scale=512 ** -0.5)
    kv = torch.cat([torch.einsum("td,hde->the", held[:, :512].float(), t.float()) for t in (wk, wv)], 2).to(torch.bfloat16)
    args = (kv[..., :128], held[:, 512:], kv[..., 128:])
    out, lse = lib.prompt_attn(q_out, *args, ints([0, n]), max_q_len=n)
    want = oracle.prompt_attn(values(q_out), *(values(t) for t in args), [0, n], [0, n], causal=True, scale=SCALE)
    check((out, lse), want)
    cut = 200
    o1, l1 = lib.prompt_attn(q_out[:cut], *(t[:cut] for t in args), ints([0, cut]), max_q_len=cut)
    o2, l2 = lib.prompt_attn(q_out[cut:], *args, ints([0, n - cut]), ints([0, n]), max_q_len=n - cut, max_k_len=n)
    check((torch.cat([o1, o2]), torch.cat([l1, l2])), want)
    # decode: the last token's absorbed query, its RoPE dims written behind the latent ones
    absorbed = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device="cuda")
    absorbed[0, :, :512] = torch.einsum("he,hde->hd", q_out[-1, :, :128].float(), wk.float()).to(torch.bfloat16)
    raw = oracle.norm(values(q)[-1:], values(qw), 1e-6)[..., 128:]
    lib.rope_append(None, None, None, pos[-1:], table, q=torch.from_numpy(raw).to(torch.bfloat16).cuda(), q_out=absorbed[..., 512:])
    assert torch.allclose(absorbed[0, :, 512:].float(), q_out[-1, :, 128:].float(), atol=2.0 ** -6, rtol=2.0 ** -7)
    verify = lib.verify if fmt == "bf16" else lib.verify_kv4
    lat, lse2 = verify(absorbed, pool, slots[None].contiguous(), ints([n - 1]), ints([[-1]]), max_seq_len=n - 1)
    final = torch.einsum("hd,hde->he", lat[0].float(), wv.float())
    # both paths round keys, values or absorbed queries of about unit size to bf16 on the way: 2^-8 each of scores of some units
    assert (final - out[-1].float()).abs().max() < 0.05 and (lse2[0] - lse[-1]).abs().max() < 0.05
