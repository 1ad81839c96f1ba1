"""GPU parity of mla_rope_append (include/mla_prompt.h) with its float64 definition.

Tolerance, per element: one rounding to bf16 (2^-8 of the value at most), and float32 arithmetic before it: the sum of
squares (at most 512 terms, added pairwise over lanes), its reciprocal root and three products stay within 2^-18 of the
value, a turned dim within 2^-20 of |x c| + |y s|. What is copied or quantised is compared exactly.
"""
import numpy as np
import pytest

import oracle
from _helpers import bf16_dev, to_dev
from speculative_decode_mla_gb300 import workloads as W

pytestmark = pytest.mark.gpu

NPOS = 5000


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()
    oracle.build()


def host_bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def values(t):
    return t.double().cpu().numpy()


def cos_sin(rng, n=NPOS):
    a = rng.uniform(0, 2 * np.pi, (n, 32))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def bf16_of(rng, *shape, scale=1.0):
    import torch
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def close(got, want, turned):
    """got (bf16 values) against want; `turned`: the same with |x|, |c|, |s| in place of the factors."""
    off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -18 * np.abs(want) + 2.0 ** -20 * turned + 1e-37)
    assert off.max() <= 0, off.max()


def check(x, q, t, w, qw, eps, halves, rows_out, q_out):
    mag = lambda f, v, weight: f(np.abs(v), np.concatenate([np.abs(t[:, :32]), np.abs(t[:, 32:])], 1), weight, eps, halves)
    plus = lambda f, v, weight: np.maximum(mag(f, v, weight), mag_minus(f, v, weight))

    def mag_minus(f, v, weight):  # |x c| + |y s| for both dims of a pair
        s = np.concatenate([np.abs(t[:, :32]), -np.abs(t[:, 32:])], 1)
        return np.abs(f(np.abs(v), s, weight, eps, halves))
    if rows_out is not None:
        close(values(rows_out), oracle.rope_rows(x, t, w, eps, halves), plus(oracle.rope_rows, x, None if w is None else np.abs(w)))
    if q_out is not None:
        close(values(q_out), oracle.rope_heads(q, t, qw, eps, halves), plus(oracle.rope_heads, q, None if qw is None else np.abs(qw)))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("n,heads,dim,width,fmt,normed", [
    (1, 1, 64, 576, "bf16", True), (1, 64, 64, 584, "kv4", True), (2, 3, 72, 576, "bf16", False), (15, 5, 128, 2112, "kv4", False),
    (16, 7, 136, 576, "bf16", True), (17, 16, 192, 592, "bf16", True), (33, 1, 256, 576, "kv4", True), (1003, 9, 192, 576, "bf16", True),
    (61, 128, 80, 2112, "none", True), (130, 0, 64, 576, "bf16", True), (4099, 2, 64, 576, "kv4", False), (257, 4, 248, 576, "bf16", False),
])
def test_rows_heads_and_pool(n, heads, dim, width, fmt, normed, halves):
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(n * 1000 + dim + halves)
    wide = bf16_of(rng, n, width, scale=2.0)
    x = wide[:, :576] if width == 576 else wide[:, 8:584] if width > 584 else wide[:, :576]
    table = cos_sin(rng)
    pos = rng.integers(0, NPOS, n).astype(np.int32)
    pos[0], pos[-1] = NPOS - 1, 0
    w = bf16_of(rng, 512) if normed else None
    q = bf16_of(rng, n, heads, dim) if heads else None
    qw = bf16_of(rng, dim) if heads and normed else None
    slots = rng.permutation(n + 40)[:n].astype(np.int32)
    slots[n // 2::5] = -1
    pool = None
    if fmt != "none":
        pool = torch.full((n + 40, 576), 7.0, dtype=torch.bfloat16, device="cuda") if fmt == "bf16" else \
            torch.full((n + 40, 416), 77, dtype=torch.uint8, device="cuda")
    before = None if pool is None else pool.clone()
    rows_out, q_out = m.rope_append(pool, x, None if pool is None else to_dev(slots), to_dev(pos), to_dev(table), weight=w, eps=1e-5, q=q,
                                    q_weight=qw, halves=halves)
    torch.cuda.synchronize()
    t = table[pos].astype(np.float64)
    check(values(x), None if q is None else values(q), t, None if w is None else values(w), None if qw is None else values(qw), 1e-5, halves,
          rows_out, q_out)
    if pool is None:
        return
    kept = slots >= 0
    expect = before.clone()
    at = torch.from_numpy(slots[kept].astype(np.int64)).cuda()
    if fmt == "bf16":
        expect[at] = rows_out[torch.from_numpy(kept).cuda()]
    else:
        expect[at] = to_dev(oracle.kv4_quantise(host_bits(rows_out)[kept]))
    assert torch.equal(pool.view(torch.uint8), expect.view(torch.uint8))


@pytest.mark.parametrize("dim", [64, 192])
@pytest.mark.parametrize("halves", [False, True])
def test_in_place_and_strided_results_are_the_same_bits(dim, halves):
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(dim)
    n, heads = 77, 6
    rows, q = bf16_of(rng, n, 576), bf16_of(rng, n, heads, dim)
    pos, table = to_dev(rng.integers(0, NPOS, n).astype(np.int32)), to_dev(cos_sin(rng))
    kw = dict(weight=bf16_of(rng, 512), halves=halves)
    for qw in (None, bf16_of(rng, dim)):
        r0, q0 = m.rope_append(None, rows, None, pos, table, q=q, q_weight=qw, **kw)
        r1, q1 = rows.clone(), q.clone()
        m.rope_append(None, r1, None, pos, table, q=q1, q_weight=qw, rows_out=r1, q_out=q1, **kw)
        assert torch.equal(r0, r1) and torch.equal(q0, q1)
        # heads before tokens in memory, and behind other dims
        wide = torch.full((heads, n, dim + 40), 3.0, dtype=torch.bfloat16, device="cuda")
        src = torch.full((n, heads, dim + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        src[..., 8:] = q
        view = wide.transpose(0, 1)[..., 32:32 + dim]
        _, q2 = m.rope_append(None, None, None, pos, table, q=src[..., 8:], q_weight=qw, q_out=view, halves=halves)
        assert q2 is view and torch.equal(view, q0)
        assert (wide[..., :32] == 3).all() and (wide[..., 32 + dim:] == 3).all()
    assert m.rope_append(None, None, None, pos, table, q=q)[0] is None


def test_padding_rows_and_bad_values_are_skipped_and_reported():
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(5)
    n = 40
    rows, q, table = bf16_of(rng, n, 576), bf16_of(rng, n, 3, 64), to_dev(cos_sin(rng))
    pos, slots = rng.integers(0, NPOS, n).astype(np.int32), np.arange(n, dtype=np.int32)
    pos[[3, 7, 9]] = [-1, NPOS, -5]
    slots[[4, 8, 10]] = [-1, n, -2]
    for fmt, bits in ((dict(), 0), (dict(debug=True), m.CHECK_BAD_POSITION | m.CHECK_BAD_SLOT)):
        pool = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        ro, qo = torch.full_like(rows, 5.0), torch.full_like(q, 5.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.rope_append(pool, rows, to_dev(slots), to_dev(pos), table, q=q, rows_out=ro, q_out=qo, dev_status=status, **fmt)
        assert int(status) == bits
        skipped = torch.zeros(n, dtype=torch.bool, device="cuda")
        skipped[[3, 7, 9]] = True
        assert (ro[skipped] == 5).all() and (qo[skipped] == 5).all() and (pool[skipped] == 7).all()
        unput = skipped.clone()
        unput[[4, 8, 10]] = True
        assert (pool[unput] == 7).all() and torch.equal(pool[~unput], ro[~unput]) and not (ro[~skipped] == 5).all(1).any()
    # positions alone, of the query heads
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.rope_append(None, None, None, to_dev(pos), table, q=q, debug=True, dev_status=status)
    assert int(status) == m.CHECK_BAD_POSITION


def test_no_rows_at_all():
    import torch
    import speculative_decode_mla_gb300 as m
    i32 = torch.zeros(0, dtype=torch.int32, device="cuda")
    pool = torch.full((3, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    r, q = m.rope_append(pool, torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda"), i32, i32, torch.zeros(1, 64, device="cuda"),
                         q=torch.zeros(0, 4, 192, dtype=torch.bfloat16, device="cuda"))
    assert r.shape == (0, 576) and q.shape == (0, 4, 192) and (pool == 7).all()


def test_wrapper_refuses():
    import torch
    import speculative_decode_mla_gb300 as m
    b, f, i = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda"), dict(dtype=torch.int32, device="cuda")
    rows, pos, table, q = torch.zeros(4, 576, **b), torch.zeros(4, **i), torch.zeros(8, 64, **f), torch.zeros(4, 2, 192, **b)
    pool, slots = torch.zeros(9, 576, **b), torch.zeros(4, **i)
    good = dict(pool=pool, rows=rows, slot_map=slots, positions=pos, cos_sin=table)
    m.rope_append(**good)
    for bad in (dict(rows=rows.float()), dict(rows=rows[:, ::2]), dict(rows=rows[:3]), dict(positions=pos.long()), dict(cos_sin=table.double()),
                dict(cos_sin=table[:, :32]), dict(slot_map=None), dict(slot_map=slots[:2]), dict(pool=None), dict(pool=pool.float()),
                dict(pool=torch.zeros(9, 400, dtype=torch.uint8, device="cuda")), dict(rows=None), dict(weight=torch.zeros(512, **f)),
                dict(weight=torch.zeros(64, **b)), dict(q=q[:2]), dict(q=q.half()), dict(q=q, q_weight=torch.zeros(64, **b)),
                dict(q_weight=torch.zeros(192, **b)), dict(q=q, q_out=q[:, :1]), dict(rows_out=rows[:2]), dict(q=q[0]),
                dict(dev_status=torch.zeros(1, device="cuda")), dict(stream=torch.cuda.Stream(), rows=rows.cpu())):
        with pytest.raises(ValueError):
            m.rope_append(**{**good, **bad})
    for bad in (dict(q=torch.zeros(4, 2, 100, **b)), dict(q=torch.zeros(4, 2, 56, **b)), dict(q=torch.zeros(4, 2, 264, **b)), dict(eps=-1.0),
                dict(rows=torch.zeros(4, 577, **b)[:, 1:]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1), q_out=None, eps=float("nan")),
                dict(debug=True)):
        with pytest.raises(m.MLAError):
            m.rope_append(**{**good, **bad})


def test_captured_on_another_stream_and_replayed():
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(8)
    n = 50
    rows, q, table = bf16_of(rng, n, 576), bf16_of(rng, n, 4, 192), to_dev(cos_sin(rng))
    pos, slots = to_dev(rng.integers(0, NPOS, n).astype(np.int32)), to_dev(rng.permutation(n).astype(np.int32))
    pool, ro, qo = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(rows), torch.zeros_like(q)
    w = bf16_of(rng, 512)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.rope_append(pool, rows, slots, pos, table, weight=w, q=q, rows_out=ro, q_out=qo, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.rope_append(pool, rows, slots, pos, table, weight=w, q=q, rows_out=ro, q_out=qo)
    rows.copy_(bf16_of(rng, n, 576))
    pos.copy_(to_dev(rng.integers(0, NPOS, n).astype(np.int32)))
    pool.zero_()
    g.replay()
    torch.cuda.synchronize()
    r1, q1 = m.rope_append(None, rows, None, pos, table, weight=w, q=q)
    assert torch.equal(ro, r1) and torch.equal(qo, q1) and torch.equal(pool[slots.long()], r1)
