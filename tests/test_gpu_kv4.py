"""GPU parity of the 4-bit pool's operators (include/mla_kv4.h) and of mla_slot_map_build with their oracles.

Integer and copy work, and the values that codes and scales stand for, are compared exactly. Attention goes against the
float64 oracle over the values that the pool stands for (bf16 numbers), with tolerances counted from its roundings.
"""
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
    oracle.build()


def host_bf16(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def same_values(got, want):
    """float64 arrays: equal, or both NaN."""
    return ((got == want) | (np.isnan(got) & np.isnan(want))).all()


# --------------------------------------------------------------------------------- append and gather

def odd_rows(n, seed):
    """bf16 bits [n, 576]: normal rows of several sizes, then blocks of zeros, ties, tiny and huge values, NaN, infinities."""
    rng = np.random.default_rng(seed)
    bits = W.normal_bf16(seed, n * 576).reshape(n, 576)
    x = W.bf16_bits_to_f32(bits).copy()
    x *= np.exp2(rng.integers(-12, 12, size=(n, 1))).astype(np.float32)
    kind = rng.integers(0, 12, size=(n, 32))
    ties = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 2, dtype=np.float32)
    for r, g in zip(*np.nonzero(kind < 6)):
        at = slice(16 * g, 16 * g + 16)
        k = kind[r, g]
        if k == 0:
            x[r, at] = 0
        elif k == 1:   # a scale of 1 + i/8 times a power of two, and values on every midpoint
            x[r, at] = ties * np.float32((1 + (g % 8) / 8) * 2.0 ** (g % 5 - 2)) * np.where(np.arange(16) < 8, 1, -1)
        elif k == 2:
            x[r, at] *= np.float32(2.0 ** -14)
        elif k == 3:
            x[r, at] = np.float32(3e38) * np.where(np.arange(16) % 3, 1, -1)
        elif k == 4:
            x[r, 16 * g + r % 16] = np.nan if g % 2 else -np.inf
        elif k == 5:
            x[r, at] = np.where(np.arange(16) % 2, -0.0, 1e-40)
    return W.f32_to_bf16_bits(x).reshape(n, 576)


@pytest.mark.parametrize("seed", range(3))
def test_append_writes_exactly_the_defined_bytes(seed):
    """Every byte of a row, the sign of values that round to zero among them."""
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(700, 576)) * np.exp2(rng.integers(-14, 14, size=(700, 1)))).astype(np.float32)
    x[:, 16:512:16] *= np.float32(2.0 ** 12)                          # the rest of a block far below its largest value
    bits = np.concatenate([odd_rows(700, 40 + seed).reshape(700, 576), W.f32_to_bf16_bits(x).reshape(700, 576)])
    pool = torch.zeros(1400, 416, dtype=torch.uint8, device="cuda")
    m.kv4_append(pool, bf16_dev(bits), torch.arange(1400, dtype=torch.int32, device="cuda"))
    assert np.array_equal(pool.cpu().numpy(), oracle.kv4_quantise(bits))


@pytest.mark.parametrize("n,width", [(1, 576), (2, 584), (15, 1152), (16, 576), (17, 592), (1003, 576)])
def test_append_then_gather_equals_the_definition(n, width):
    import torch
    import speculative_decode_mla_gb300 as m
    bits = odd_rows(n, 40 + n)
    wide = np.full((n, width), 0x7F81, dtype=np.uint16)    # what lies beside the rows is not read as a dim
    wide[:, :576] = bits
    rng = np.random.default_rng(n)
    slots = rng.permutation(n + 9)[:n].astype(np.int32)
    slots[rng.random(n) < 0.2] = -1
    before = rng.integers(0, 256, size=(n + 9, 416), dtype=np.uint8)
    want = before.copy()
    want[slots[slots >= 0]] = oracle.kv4_quantise(bits)[slots >= 0]
    pool = to_dev(before)
    m.kv4_append(pool, bf16_dev(wide)[:, :576], to_dev(slots))
    got = pool.cpu().numpy()
    untouched = np.setdiff1d(np.arange(n + 9), slots)
    assert np.array_equal(got[untouched], before[untouched])
    assert np.array_equal(got[:, 256:], want[:, 256:])       # scales and RoPE dims, to the bit
    kept = slots[slots >= 0]
    assert same_values(oracle.kv4_values(got[kept]), oracle.kv4_values(want[kept]))
    out = m.kv4_gather(pool, to_dev(slots))
    torch.cuda.synchronize()
    values = W.bf16_bits_to_f32(host_bf16(out)).astype(np.float64)
    assert same_values(values[slots >= 0], oracle.kv4_values(want[kept]))
    assert (host_bf16(out)[slots < 0] == 0).all()


def test_gather_reads_every_code_and_scale_and_repeated_slots():
    import torch
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(3)
    rows = rng.integers(0, 256, size=(300, 416), dtype=np.uint8)
    rows[:256, 256:288] = np.arange(256, dtype=np.uint8)[:, None]
    slots = np.concatenate([np.arange(300), rng.integers(0, 300, 700)]).astype(np.int32)
    out = m.kv4_gather(to_dev(rows), to_dev(slots))
    torch.cuda.synchronize()
    values = W.bf16_bits_to_f32(host_bf16(out)).astype(np.float64)
    assert same_values(values, oracle.kv4_values(rows[slots]))


def test_bad_slots_are_reported_and_skipped():
    import torch
    import speculative_decode_mla_gb300 as m
    bits = W.normal_bf16(6, 5 * 576).reshape(5, 576)
    slots = np.array([2, 7, -2, 0, 1 << 30], dtype=np.int32)
    pool = torch.zeros(7, 416, dtype=torch.uint8, device="cuda")
    for debug in (False, True):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.kv4_append(pool, bf16_dev(bits), to_dev(slots), debug=debug, dev_status=st)
        assert st.item() == (m.CHECK_BAD_SLOT if debug else 0)
        st.zero_()
        out = m.kv4_gather(pool, to_dev(slots), debug=debug, dev_status=st)
        assert st.item() == (m.CHECK_BAD_SLOT if debug else 0)
    got = pool.cpu().numpy()
    want = oracle.kv4_quantise(bits)
    assert same_values(oracle.kv4_values(got[[2, 0]]), oracle.kv4_values(want[[0, 3]]))
    assert (got[[1, 3, 4, 5, 6]] == 0).all()
    assert (host_bf16(out)[[1, 2, 4]] == 0).all()


def test_no_rows():
    import torch
    import speculative_decode_mla_gb300 as m
    pool = torch.zeros(3, 416, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    m.kv4_append(pool, torch.empty(0, 576, dtype=torch.bfloat16, device="cuda"), none)
    assert m.kv4_gather(pool, none).shape == (0, 576) and not pool.any()


def test_python_refusals():
    import torch
    import speculative_decode_mla_gb300 as m
    pool = torch.zeros(8, 416, dtype=torch.uint8, device="cuda")
    rows = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    for args in ((pool[:, :400], rows, slots), (pool.to(torch.int8), rows, slots), (pool, rows.float(), slots),
                 (pool, rows, slots.long()), (pool, rows, slots[:3]), (pool, rows[:, :512], slots), (pool, rows.cpu(), slots),
                 (pool, rows.t().contiguous().t(), slots), (pool, rows, slots.cpu())):
        with pytest.raises(ValueError):
            m.kv4_append(*args)
    with pytest.raises(m.MLAError):          # row stride not a multiple of 8
        m.kv4_append(pool, torch.zeros(4, 577, dtype=torch.bfloat16, device="cuda")[:, :576], slots)
    with pytest.raises(ValueError):
        m.kv4_gather(pool, slots, out=torch.empty(4, 576, device="cuda"))
    q = torch.zeros(4, 2, 576, dtype=torch.bfloat16, device="cuda")
    table, lens, par = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 16), (2,), (2, 2)))
    good = dict(max_seq_len=8)
    m.verify_kv4(q, pool, table, lens, par, **good)
    for bad in (dict(q=q[:2]), dict(q=q.float()), dict(pool=rows), dict(slot_table=table.long()), dict(slot_table=table[:1]),
                dict(seq_lens=lens[:1]), dict(tree_parent=par.t())):
        a = dict(q=q, pool=pool, slot_table=table, seq_lens=lens, tree_parent=par)
        a.update(bad)
        with pytest.raises(ValueError):
            m.verify_kv4(a["q"], a["pool"], a["slot_table"], a["seq_lens"], a["tree_parent"], **good)
    with pytest.raises(ValueError):
        m.verify_kv4(q, pool, table, lens, par, out=torch.empty(4, 2, 512, device="cuda"), **good)
    with pytest.raises(m.MLAError):          # the table is too narrow
        m.verify_kv4(q, pool, table, lens, par, max_seq_len=15)
    with pytest.raises(m.MLAError):          # the workspace is too small
        m.verify_kv4(q, pool, table, lens, par, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **good)


# ------------------------------------------------------------------------------------------- slot maps

def map_case(B, page, seed, hi=70, extra_pages=5, bad=False, prompt=False):
    rng = np.random.default_rng(seed)
    seq = np.zeros(B, np.int64) if prompt else rng.integers(0, hi, B)
    new = rng.integers(0, hi, B)
    new[rng.random(B) < 0.2] = 0
    held = seq + (0 if prompt else rng.integers(0, 12, B))
    if bad:
        for i, v in enumerate([(-1, 3, -1), (4, -2, 4), (9, 1, 8), (5, 10 ** 6, 5), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)]):
            seq[3 * i + 1], new[3 * i + 1], held[3 * i + 1] = v
    stride = 2 * hi + 13
    blocks = -(-stride // page)
    pages = rng.permutation(B * blocks + extra_pages).astype(np.int32)
    block = np.zeros((B, blocks), np.int32)
    table = np.full((B, stride), -9, np.int32)
    used = 0
    for b in range(B):
        h = int(held[b])
        if not 0 <= h <= stride:
            continue
        k = -(-h // page)
        block[b, :k] = pages[used:used + k]
        used += k
        t = np.arange(h)
        table[b, :h] = rng.permutation(block[b, t // page] * page + t % page)   # as accepted paths leave it
    take = sum(max(0, -(-max(int(h), int(s) + int(n)) // page) - -(-int(h) // page)) for s, n, h in zip(seq, new, held)
               if s >= 0 and n >= 0 and h >= s and max(int(h), int(s) + int(n)) <= stride)
    tokens = sum(int(n) for s, n, h in zip(seq, new, held) if s >= 0 and n >= 0 and h >= s and max(int(h), int(s) + int(n)) <= stride)
    return dict(seq=seq.astype(np.int32), new=new.astype(np.int32), held=held.astype(np.int32), page=page, num_pages=len(pages),
                free=np.concatenate([pages[used:], np.full(3, -77, np.int32)]), count=len(pages) - used, block=block, table=table,
                take=take, tokens=tokens)


def run_map(c, capacity, count=None, held=True, block=True, offset=0, debug=True):
    import torch
    import speculative_decode_mla_gb300 as m
    count = c["count"] if count is None else count
    h = c["held"] if held else None
    want = oracle.slot_map_build(c["seq"], c["new"], h, c["page"], c["num_pages"], c["free"], count,
                                 c["block"] if block else None, c["table"], capacity)
    block_d, table_d = to_dev(c["block"].copy()), to_dev(c["table"].copy())
    slot_map = torch.full((capacity + 8,), 1234567, dtype=torch.int32, device="cuda")[offset:offset + capacity]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    count_d = torch.tensor([count], dtype=torch.int32, device="cuda")
    got_map, cu, held_out, left = m.slot_map_build(
        to_dev(c["seq"]), to_dev(c["new"]), to_dev(c["free"]), count_d, table_d, page_size=c["page"], num_pages=c["num_pages"],
        held_lens=to_dev(h) if held else None, block_table=block_d if block else None, slot_map=slot_map, debug=debug, dev_status=st)
    torch.cuda.synchronize()
    w_block, w_table, w_map, w_cu, w_held, w_left, bits = want
    assert np.array_equal(got_map.cpu().numpy(), w_map)
    assert np.array_equal(table_d.cpu().numpy(), w_table)
    assert np.array_equal(block_d.cpu().numpy(), w_block if block else c["block"])
    assert np.array_equal(cu.cpu().numpy(), w_cu) and np.array_equal(held_out.cpu().numpy(), w_held)
    assert left.item() == w_left and count_d.item() == count
    flags = {"length": m.CHECK_BAD_LENGTH, "pages": m.CHECK_NO_PAGES, "slot": m.CHECK_BAD_SLOT}
    assert st.item() == (sum(flags[b] for b in bits) if debug else 0)
    return bits


@pytest.mark.parametrize("B,page,offset", [(1, 1, 0), (1, 16, 1), (5, 3, 2), (64, 1, 0), (33, 64, 3), (513, 7, 0), (1000, 16, 0),
                                           (8192, 1, 0)])
def test_slot_map_equals_the_definition(B, page, offset):
    c = map_case(B, page, 7 * B + page, hi=70 if B < 2000 else 9)
    assert run_map(c, c["tokens"] + 6, offset=offset) == set()
    assert run_map(c, c["tokens"], offset=offset) == set()
    if B < 2000:
        c = map_case(B, page, 11 * B + page, prompt=True)
        assert run_map(c, c["tokens"] + 1, held=False) == set()


def test_slot_map_pages_of_one_need_no_block_table():
    assert run_map(map_case(40, 1, 5), 40 * 70, block=False) == set()


@pytest.mark.parametrize("page", [1, 16])
def test_slot_map_refuses_as_a_whole(page):
    c = map_case(50, page, 9)
    assert c["take"] > 0
    assert run_map(c, c["tokens"], count=c["take"]) == set()
    assert run_map(c, c["tokens"], count=c["take"] - 1) == {"pages"}
    assert run_map(c, c["tokens"] - 1) == {"pages"}
    assert run_map(c, c["tokens"], count=-1) == {"pages"}
    assert run_map(c, c["tokens"], count=len(c["free"]) + 1) == {"pages"}
    assert run_map(c, c["tokens"], count=-1, debug=False) == {"pages"}
    assert run_map(c, 0) == {"pages"}


def test_slot_map_bad_lengths_pages_and_slots():
    c = map_case(30, 4, 13, bad=True)
    assert run_map(c, c["tokens"] + 2) == {"length"}
    c = map_case(30, 4, 14)
    c["free"][c["count"] - 3] = c["num_pages"]        # taken by an early sequence
    c["free"][c["count"] - 5] = -1
    c["table"][:, 3] = 1 << 29
    assert "slot" in run_map(c, c["tokens"] + 2)
    c = map_case(6, 4, 15)
    c["new"][:] = 0
    assert run_map(c, 5) == set()


def test_slot_map_long_prompts_in_pages():
    rng = np.random.default_rng(1)
    B, page = 9, 64
    new = rng.integers(20000, 30000, B).astype(np.int32)
    blocks = 30000 // page + 1
    pages = rng.permutation(B * blocks).astype(np.int32)
    c = dict(seq=np.zeros(B, np.int32), new=new, held=np.zeros(B, np.int32), page=page, num_pages=B * blocks, free=pages,
             count=len(pages), block=np.zeros((B, blocks), np.int32), table=np.zeros((B, 30001), np.int32))
    assert run_map(c, int(new.sum()) + 1000) == set()


# ------------------------------------------------------------------------------------------- attention

def random_pool(n, seed, lat=1.0):
    """(rows uint8 [n, 416], the bf16 bits of their values)."""
    x = W.bf16_bits_to_f32(W.normal_bf16(seed, n * 576)).reshape(n, 576).copy()
    x[:, :512] *= np.linspace(0.3, 2.0, 512, dtype=np.float32) * np.float32(lat)
    rows = oracle.kv4_quantise(W.f32_to_bf16_bits(x))
    return rows, oracle.kv4_bf16(rows)


def problem(lens, T, H, seed, *, tree="random", sizes=None, lat=1.0, slack=7):
    p = W.custom_problem(lens, T, H, tree=tree, seed=seed, pool_slack=slack, stride_pad=3)
    rows, bits = random_pool(p.num_slots, 1000 + seed, lat)
    return p, rows, bits


def expect(p, bits, q=None, sizes=None, parents=None, scale=W.SOFTMAX_SCALE):
    """(out, lse) of the oracle; padding nodes give 0 and -inf."""
    q = p.q if q is None else q
    parents = p.tree_parent if parents is None else parents
    if sizes is None:
        o, l = oracle.verify(p.seq_lens, p.slot_table, parents, q, bits, num_heads=p.H, scale=scale)
        return o.reshape(p.rows, 512), l
    out, lse = np.zeros((p.B, p.T * p.H, 512)), np.full((p.B, p.T * p.H), -np.inf)
    q = q.reshape(p.B, p.T, p.H, 576)
    for b in range(p.B):
        t = int(sizes[b])
        o, l = oracle.verify(p.seq_lens[b:b + 1], p.slot_table[b:b + 1], parents[b:b + 1, :t], q[b, :t], bits,
                             num_heads=p.H, scale=scale)
        out[b, :t * p.H], lse[b, :t * p.H] = o.reshape(-1, 512), l
    return out.reshape(p.rows, 512), lse.reshape(-1)


def call(p, rows, q=None, sizes=None, parents=None, table=None, **kw):
    import torch
    import speculative_decode_mla_gb300 as m
    out, lse = m.verify_kv4(bf16_dev(p.q if q is None else q), to_dev(rows), to_dev(p.slot_table if table is None else table),
                            to_dev(p.seq_lens), to_dev(p.tree_parent if parents is None else parents),
                            max_seq_len=kw.pop("max_seq_len", p.max_seq_len),
                            tree_sizes=None if sizes is None else to_dev(np.asarray(sizes, np.int32)), **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().reshape(p.rows, 512).astype(np.float64), lse.cpu().numpy().reshape(-1).astype(np.float64)


def assert_close(got, want, q, bits, scale=W.SOFTMAX_SCALE, f32=False):
    """Per element of out, relative to the largest value a row can see: a weight is rounded to fp16 once (2^-11), a split's output
    to fp16 once (2^-11), the result to bf16 once (2^-8); a score is a sum of 576 products in fp32, so it is off by at most
    576 * 2^-24 of the sum of their magnitudes, which moves every weight and the lse by as much (weights: twice, with the norm)."""
    (o, l), (wo, wl) = got, want
    assert np.array_equal(np.isnan(wo), np.isnan(o)) and np.array_equal(np.isneginf(wl), np.isneginf(l))
    fine = np.isfinite(wl)
    v = W.bf16_bits_to_f32(bits).astype(np.float64)
    v = v[np.isfinite(v).all(axis=1)]
    qs = np.abs(W.bf16_bits_to_f32(q).astype(np.float64)).reshape(-1, 576).max(axis=0)
    size = float((np.abs(v) @ qs).max()) * scale
    d_score = 576 * 2.0 ** -24 * size + 2.0 ** -20
    top = np.abs(v[:, :512]).max()
    tol = (2.0 ** -11 + 2.0 ** -11 + (0 if f32 else 2.0 ** -8) + 2 * d_score) * top
    err = np.abs(o[fine] - wo[fine]).max() if fine.any() else 0.0
    lerr = np.abs(l[fine] - wl[fine]).max() if fine.any() else 0.0
    rel = np.linalg.norm(o[fine] - wo[fine]) / max(np.linalg.norm(wo[fine]), 1e-300) if fine.any() else 0.0
    assert err <= tol, f"max error {err:.3e}, allowed {tol:.3e}"
    assert rel <= 5e-3, f"relative error {rel:.3e}"
    assert lerr <= d_score + 2.0 ** -22 * (1 + np.abs(wl[fine]).max() if fine.any() else 1), f"lse error {lerr:.3e}, allowed {d_score:.3e}"
    return err, lerr


SHAPES = [([1], 1, 1), ([0], 1, 1), ([0], 64, 3), ([63], 1, 16), ([64], 2, 1), ([127], 1, 128), ([128], 1, 129), ([129], 5, 7),
          ([1000], 8, 8), ([3000], 16, 8), ([0, 1, 63, 64, 65, 127, 128, 129, 500, 2049], 3, 11), ([700, 90, 5000], 9, 13),
          ([4100], 64, 8), ([255, 256], 33, 4), ([10, 2000, 300, 40, 5] * 14, 2, 3)]


@pytest.mark.parametrize("simt", [True, False], ids=["simt", "default"])
@pytest.mark.parametrize("lens,T,H", SHAPES, ids=[f"{len(s[0])}x{max(s[0])}T{s[1]}H{s[2]}" for s in SHAPES])
def test_verify_matches_the_oracle(lens, T, H, simt):
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem(lens, T, H, 300 + len(lens) + T)
    got = call(p, rows, flags=m.MLA_FLAG_SIMT if simt else None, out_dtype=m.MLA_DTYPE_F32)
    assert_close(got, expect(p, bits), p.q, bits, f32=True)


@pytest.mark.parametrize("splits", [0, 1, 2, 7, 1000])
@pytest.mark.parametrize("tree", ["chain", "star"])
def test_verify_splits_and_trees(splits, tree):
    p, rows, bits = problem([2500, 131], 12, 5, 41, tree=tree)
    assert_close(call(p, rows, num_splits=splits), expect(p, bits), p.q, bits)


@pytest.mark.parametrize("hint", [0, 1, 4000, 10 ** 9])
def test_verify_ragged_trees_and_hints(hint):
    p, rows, bits = problem([900, 0, 33, 2048, 7], 9, 15, 42)
    sizes = [9, 1, 4, 8, 2]
    got = call(p, rows, sizes=sizes, total_tokens_hint=hint)
    want = expect(p, bits, sizes=sizes)
    assert_close(got, want, p.q, bits)
    pad = np.isneginf(want[1])
    assert pad.any() and (got[0][pad] == 0).all()


MANY = [int(x) for x in np.random.default_rng(5).integers(0, 900, size=100)]


@pytest.mark.parametrize("lens,T,H,kw", [
    (MANY, 2, 9, {}), (MANY, 2, 9, dict(num_splits=1)), (MANY, 2, 9, dict(num_splits=3, total_tokens_hint=1)),
    ([900, 0, 3000, 1500], 16, 20, {}), ([900, 0, 3000, 1500], 16, 20, dict(num_splits=1)),
    ([900, 0, 3000, 1500], 16, 20, dict(num_splits=2)), ([900, 0, 3000, 1500], 16, 20, dict(total_tokens_hint=10 ** 9)),
    ([5] * 33 + [6000], 5, 29, {}), ([5] * 33 + [6000], 5, 29, dict(num_splits=1)), ([0] * 70, 1, 17, {}),
    ([200, 1] * 80, 1, 20, dict(total_tokens_hint=300)),
], ids=lambda x: str(len(x)) if isinstance(x, list) else None)
def test_verify_shares_that_begin_inside_a_sequence(lens, T, H, kw):
    """A pair of CTAs takes a run of tiles that may hold several sequences and row tiles, whole or in part."""
    p, rows, bits = problem(lens, T, H, 500 + len(lens))
    assert_close(call(p, rows, **kw), expect(p, bits), p.q, bits)
    sizes = 1 + np.arange(p.B) % T
    assert_close(call(p, rows, sizes=sizes, **kw), expect(p, bits, sizes=sizes), p.q, bits)


@pytest.mark.parametrize("n", [0, 1, 500, 4000, 9600, 9727, 9728, 9729, 20000])
def test_verify_lengths_far_below_the_limit(n):
    """One captured call with room for 150,000 positions, replayed for shorter sequences (76 pairs x 128 positions are 9728)."""
    import torch
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem([20000], 4, 8, 700)
    room = 150000
    table = np.zeros((1, room + 4), np.int32)
    lens = torch.full((1,), room, dtype=torch.int32, device="cuda")
    dev = (bf16_dev(p.q), to_dev(rows), to_dev(table), lens, to_dev(p.tree_parent))
    m.verify_kv4(*dev, max_seq_len=room)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = m.verify_kv4(*dev, max_seq_len=room, out_dtype=m.MLA_DTYPE_F32)
    table[0, :n + 4] = p.slot_table[0, :n + 4]
    dev[2].copy_(to_dev(table))
    lens.fill_(n)
    g.replay()
    torch.cuda.synchronize()
    want = oracle.verify(np.array([n], np.int32), table, p.tree_parent, p.q, bits, num_heads=8, scale=W.SOFTMAX_SCALE)
    got = (out.cpu().numpy().reshape(-1, 512).astype(np.float64), lse.cpu().numpy().reshape(-1).astype(np.float64))
    assert_close(got, (want[0].reshape(-1, 512), want[1]), p.q, bits, f32=True)


@pytest.mark.parametrize("B,T,H", [(33, 1, 3), (33, 1, 17), (64, 2, 9), (65, 1, 17), (65, 1, 3), (1000, 1, 17), (3000, 2, 9), (3000, 2, 3)])
def test_verify_many_short_sequences(B, T, H):
    """More sequences than a warp has lanes, most of them one tile: both kernels over the same rows."""
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(B)
    lens = [int(x) for x in np.where(rng.random(B) < 0.8, rng.integers(0, 100, B), rng.integers(100, 700, B))]
    p, rows, bits = problem(lens, T, H, 600 + B)
    got, ref = call(p, rows, out_dtype=m.MLA_DTYPE_F32), call(p, rows, out_dtype=m.MLA_DTYPE_F32, flags=m.MLA_FLAG_SIMT)
    assert_close(got, ref, p.q, bits, f32=True)
    if B <= 65:
        assert_close(got, expect(p, bits), p.q, bits, f32=True)


FEW = [0, 1, 31, 32, 33, 63, 64, 65, 100, 300, 1000, 127, 128, 129, 5, 2500, 17, 700]


@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (16, 1), (2, 8), (3, 5), (5, 3)])
@pytest.mark.parametrize("kw", [{}, dict(num_splits=1), dict(num_splits=9), dict(total_tokens_hint=1)], ids=["plan", "one", "nine", "hint"])
def test_verify_few_rows(T, H, kw):
    """At most 16 rows a sequence and many sequences: the kernel for few rows."""
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem(FEW, T, H, 800 + T)
    d = m.make_desc(p.B, T, H, p.num_slots, p.slot_table.shape[1], p.max_seq_len)
    assert m.kv4_plan(d, 152).kernel == 2
    assert_close(call(p, rows, out_dtype=m.MLA_DTYPE_F32, **kw), expect(p, bits), p.q, bits, f32=True)
    sizes = 1 + np.arange(p.B) % T
    got, want = call(p, rows, sizes=sizes, **kw), expect(p, bits, sizes=sizes)
    assert_close(got, want, p.q, bits)
    assert (got[0][np.isneginf(want[1])] == 0).all()


def test_verify_few_rows_of_any_size_with_nan_and_infinities():
    p, rows, bits = problem(FEW, 4, 4, 810)
    x = W.bf16_bits_to_f32(p.q).copy()
    x[0::4] *= np.float32(2.0 ** -100)
    x[1::4] *= np.float32(8)
    x[2::4, :, :512] *= np.float32(2.0 ** -25)
    x[3::4] = 0
    q = W.f32_to_bf16_bits(x).reshape(p.q.shape)
    want = expect(p, bits, q=q)
    assert_close(call(p, rows, q=q), want, q, bits)
    bad = rows.copy()
    parents = np.tile(np.array([-1, 0, 0, 2], np.int32), (p.B, 1))
    want = expect(p, bits, parents=parents)
    clean = np.ones(p.rows, bool)
    for b in (3, 10):
        bad[p.slot_table[b, p.seq_lens[b] + 1], 256 + 7] = 0x7F       # node 1: NaN in a block; only node 1 sees it
        bad[p.slot_table[b, p.seq_lens[b] + 2], 288:].view(np.uint16)[:] = 0x7F80   # node 2: infinite RoPE dims (2 and 3)
        clean[(b * 4 + 1) * 4:(b * 4 + 4) * 4] = False
    bad[p.slot_table[15, 700], 256] = 0xFF                            # a prefix position of one sequence
    clean[15 * 16:16 * 16] = False
    o, l = call(p, bad, parents=parents)
    assert_close((o[clean], l[clean]), (want[0][clean], want[1][clean]), p.q, bits)
    s, sl = call(p, bad, parents=parents, flags=2)
    assert np.isnan(l[~clean]).all() and np.array_equal(np.isnan(s), np.isnan(o))


def test_verify_few_rows_checks_slots_and_repeatability():
    import torch
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem(FEW, 2, 8, 820)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=m.MLA_FLAG_DEBUG_CHECKS, dev_status=st)
    a = call(p, rows, **kw)
    perm = np.random.default_rng(1).permutation(p.num_slots)
    moved = np.empty_like(rows)
    moved[perm] = rows
    b = call(p, moved, table=perm[p.slot_table].astype(np.int32))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    table, parents = p.slot_table.copy(), p.tree_parent.copy()
    table[15, 2400] = -7
    parents[17, 1] = 1
    for bad, flag in ((dict(table=table), m.CHECK_BAD_SLOT), (dict(parents=parents), m.CHECK_BAD_PARENT),
                      (dict(max_seq_len=2499), m.CHECK_BAD_LENGTH), (dict(sizes=[3] * p.B), m.CHECK_BAD_LENGTH)):
        with pytest.raises(m.MLAError):
            call(p, rows, **kw, **bad)
        assert st.item() == flag


def test_debug_checks_of_the_last_sequences():
    """Bad slots and parents that only a cluster's later sequences hold are reported too."""
    import torch
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem(MANY, 2, 9, 51)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=m.MLA_FLAG_DEBUG_CHECKS, dev_status=st, num_splits=1)
    assert_close(call(p, rows, **kw), expect(p, bits), p.q, bits)
    for b in (1, 50, 99):
        table, parents = p.slot_table.copy(), p.tree_parent.copy()
        table[b, p.seq_lens[b]] = -1
        parents[b, 1] = 1
        for bad, flag in ((dict(table=table), m.CHECK_BAD_SLOT), (dict(parents=parents), m.CHECK_BAD_PARENT)):
            with pytest.raises(m.MLAError):
                call(p, rows, **kw, **bad)
            assert st.item() == flag


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** -6, 1.0, 8.0])
def test_verify_queries_of_any_size(size):
    """Rows of very different sizes in one tile, up to scores that let one key take all the weight."""
    p, rows, bits = problem([1500], 4, 8, 43)
    x = W.bf16_bits_to_f32(p.q).copy()
    x[0] *= np.float32(size)
    x[1] *= np.float32(2.0 ** -30)
    x[2, :, :512] *= np.float32(2.0 ** -25)       # the RoPE dims carry the score
    x[3] = 0
    q = W.f32_to_bf16_bits(x).reshape(p.q.shape)
    assert_close(call(p, rows, q=q), expect(p, bits, q=q), q, bits)


@pytest.mark.parametrize("lat", [2.0 ** -8, 300.0])
def test_verify_latents_of_any_size(lat):
    p, rows, bits = problem([700], 2, 4, 44, lat=lat)
    x = W.bf16_bits_to_f32(p.q).copy() / np.float32(max(1.0, lat))
    q = W.f32_to_bf16_bits(x).reshape(p.q.shape)
    assert_close(call(p, rows, q=q), expect(p, bits, q=q), q, bits)


def test_verify_many_small_weights_beside_a_large_one():
    """One key far above 20,000 others: their weights are small, their sum is not."""
    p, rows, bits = problem([20000], 1, 2, 45)
    x = np.zeros((1, 2, 576), dtype=np.float32)
    x[:, :, 512] = 16.0
    k = oracle.kv4_values(rows)
    r = rows.copy()
    rope = np.zeros((len(r), 64), dtype=np.float32)
    rope[p.slot_table[0, 777], 0] = 9.0            # score 16 * 9 / sqrt(192) = 10.4; e^10.4 is 32,860
    r[:, 288:] = W.f32_to_bf16_bits(rope).reshape(len(r), 64).view(np.uint8)
    bits = oracle.kv4_bf16(r)
    q = W.f32_to_bf16_bits(x).reshape(p.q.shape)
    assert_close(call(p, r, q=q), expect(p, bits, q=q), q, bits)
    assert k.shape == (len(r), 576)


def test_a_key_with_nan_reaches_only_the_rows_that_see_it():
    """A NaN scale in a tree node's row, and infinities in other nodes' RoPE dims: nodes that do not see them are as if they were not there."""
    p, rows, bits = problem([200], 6, 3, 46)
    parents = np.array([[-1, 0, 0, -1, 3, 4]], dtype=np.int32)
    bad = rows.copy()
    bad[p.slot_table[0, 200 + 2], 256 + 5] = 0x7F                     # node 2: NaN in a block
    rope = bad[p.slot_table[0, 200 + 4], 288:].view(np.uint16)
    rope[:] = 0x7F80                                                  # node 4: infinite RoPE dims (nodes 4 and 5 see it)
    want = expect(p, bits, parents=parents)
    o, l = call(p, bad, parents=parents)
    node = np.arange(p.rows) // p.H
    clean = np.isin(node, [0, 1, 3])
    assert_close((o[clean], l[clean]), (want[0][clean], want[1][clean]), p.q, bits)
    assert np.isnan(o[node == 2]).all() and np.isnan(l[node == 2]).all()
    s, _ = call(p, bad, parents=parents, flags=2)
    assert np.array_equal(np.isnan(s), np.isnan(o))


def test_nan_in_a_prefix_and_in_unread_slots():
    p, rows, bits = problem([150, 90], 2, 2, 47)
    used = np.concatenate([p.slot_table[b, :p.seq_lens[b] + p.T] for b in range(2)])
    bad = rows.copy()
    spare = np.setdiff1d(np.arange(p.num_slots), used)
    bad[spare] = 0xFF                                                 # rows that no sequence holds: all NaN
    want = expect(p, bits)
    got = call(p, bad)
    assert_close(got, want, p.q, bits)
    bad[p.slot_table[0, 10], 256] = 0xFF                              # sequence 0's prefix
    o, l = call(p, bad)
    first = np.arange(p.rows) < p.T * p.H
    assert np.isnan(o[first]).all() and np.isnan(l[first]).all()
    assert np.array_equal(o[~first], got[0][~first]) and np.array_equal(l[~first], got[1][~first])


def test_result_does_not_depend_on_the_slots():
    p, rows, bits = problem([3000, 1234], 7, 9, 48)
    a = call(p, rows)
    perm = np.random.default_rng(0).permutation(p.num_slots)
    moved = np.empty_like(rows)
    moved[perm] = rows
    b = call(p, moved, table=perm[p.slot_table].astype(np.int32))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    c = call(p, rows)
    assert np.array_equal(a[0], c[0]) and np.array_equal(a[1], c[1])


def test_debug_checks():
    import torch
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem([300, 40], 4, 2, 49)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=m.MLA_FLAG_DEBUG_CHECKS, dev_status=st)
    assert_close(call(p, rows, **kw), expect(p, bits), p.q, bits)
    table = p.slot_table.copy()
    table[1, 20] = p.num_slots
    parents = p.tree_parent.copy()
    parents[0, 2] = 3
    for bad, flag in ((dict(table=table), m.CHECK_BAD_SLOT), (dict(parents=parents), m.CHECK_BAD_PARENT),
                      (dict(max_seq_len=299), m.CHECK_BAD_LENGTH), (dict(sizes=[4, 5]), m.CHECK_BAD_LENGTH)):
        with pytest.raises(m.MLAError) as e:
            call(p, rows, **kw, **bad)
        assert e.value.status == -5 and st.item() == flag
    st.zero_()
    o, l = call(p, rows, table=table)                                 # without the checks: clamped, no fault
    assert np.isfinite(l).all()


def test_verify_over_the_gathered_bf16_pool_agrees():
    """mla_verify_attn over what kv4_gather reads out is the same attention."""
    import torch
    import speculative_decode_mla_gb300 as m
    p, rows, bits = problem([5000], 16, 8, 50)
    pool = m.kv4_gather(to_dev(rows), torch.arange(p.num_slots, dtype=torch.int32, device="cuda"))
    o, l = m.verify(bf16_dev(p.q), pool, to_dev(p.slot_table), to_dev(p.seq_lens), to_dev(p.tree_parent),
                    max_seq_len=p.max_seq_len, out_dtype=m.MLA_DTYPE_F32)
    a = call(p, rows, out_dtype=m.MLA_DTYPE_F32)
    top = np.abs(W.bf16_bits_to_f32(bits)[:, :512]).max()
    assert np.abs(o.cpu().numpy().reshape(p.rows, 512) - a[0]).max() <= 2.0 ** -7 * top
    assert np.abs(l.cpu().numpy().reshape(-1) - a[1]).max() <= 1e-3


# -------------------------------------------------------------------------------- together, as used

def test_decode_steps_together_in_a_captured_graph():
    """Four decode steps of three requests: slots for the tree, its rows appended, attention, a path accepted. The first three calls
    are captured once and replayed with every step's lengths."""
    import torch
    import speculative_decode_mla_gb300 as m
    B, T, H, page, stride, max_len = 3, 6, 4, 4, 420, 400
    rng = np.random.default_rng(8)
    lens = np.array([130, 1, 300], np.int32)
    num_pages = 300
    free = rng.permutation(num_pages).astype(np.int32)
    pool_rows, _ = random_pool(num_pages * page, 77)
    pool_np = pool_rows.copy()
    i32 = dict(dtype=torch.int32, device="cuda")
    pool, free_d = to_dev(pool_rows), to_dev(free)
    block, table = torch.zeros(B, stride // page + 1, **i32), torch.zeros(B, stride, **i32)
    block_np, table_np = block.cpu().numpy(), table.cpu().numpy()
    count = torch.tensor([num_pages], **i32)
    # the prompts' tokens
    zero = torch.zeros(B, **i32)
    _, _, held, left = m.slot_map_build(zero, to_dev(lens), free_d, count, table, page_size=page, num_pages=num_pages,
                                        map_capacity=int(lens.sum()), block_table=block)
    block_np, table_np, _, _, held_np, left_np, bits = oracle.slot_map_build(np.zeros(B, np.int32), lens, None, page, num_pages,
                                                                             free, num_pages, block_np, table_np, int(lens.sum()))
    assert bits == set()
    seq, held_in, held_out = to_dev(lens), held.clone(), torch.empty(B, **i32)
    new = torch.full((B,), T, **i32)
    count_in, count_out = left.clone(), torch.empty(1, **i32)
    slot_map, cu = torch.empty(B * T, **i32), torch.empty(B + 1, **i32)
    rows_in = torch.empty(B * T, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(B * T, H, 576, dtype=torch.bfloat16, device="cuda")
    parents = torch.zeros(B, T, **i32)
    out = torch.empty(B * T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B * T, H, device="cuda")
    desc = m.make_desc(B, T, H, pool.shape[0], stride, max_len)
    ws = torch.empty(m.kv4_workspace_size(desc), dtype=torch.uint8, device="cuda")

    def step():
        m.slot_map_build(seq, new, free_d, count_in, table, page_size=page, num_pages=num_pages, held_lens=held_in,
                         block_table=block, slot_map=slot_map, cu_new=cu, held_out=held_out, free_left=count_out)
        m.kv4_append(pool, rows_in, slot_map)
        m.verify_kv4(q, pool, table, seq, parents, max_seq_len=max_len, out=out, lse=lse, workspace=ws)

    graph = None
    for it in range(4):
        tree = np.stack([W.random_tree(100 * it + b, T) for b in range(B)])
        bits_rows = W.normal_bf16(900 + it, B * T * 576).reshape(B * T, 576)
        bits_q = W.normal_bf16(800 + it, B * T * H * 576).reshape(B * T, H, 576)
        rows_in.copy_(bf16_dev(bits_rows))
        q.copy_(bf16_dev(bits_q))
        parents.copy_(to_dev(tree))
        if it == 0:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        block_np, table_np, map_np, cu_np, held_np, left_np, found = oracle.slot_map_build(
            lens, np.full(B, T), held_np, page, num_pages, free, left_np, block_np, table_np, B * T)
        assert found == set()
        assert np.array_equal(table.cpu().numpy(), table_np) and np.array_equal(slot_map.cpu().numpy(), map_np)
        assert np.array_equal(block.cpu().numpy(), block_np) and count_out.item() == left_np
        assert np.array_equal(held_out.cpu().numpy(), held_np)
        pool_np[map_np] = oracle.kv4_quantise(bits_rows)
        values = oracle.kv4_bf16(pool_np)
        ro, rl = oracle.verify(lens, table_np, tree, bits_q, values, num_heads=H, scale=W.SOFTMAX_SCALE)
        got = (out.float().cpu().numpy().reshape(-1, 512).astype(np.float64), lse.cpu().numpy().reshape(-1).astype(np.float64))
        assert_close(got, (ro.reshape(-1, 512), rl), bits_q, values)
        # accept a random path of each tree
        acc, n = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
        for b in range(B):
            node, path = int(rng.integers(0, T)), []
            while node >= 0:
                path.append(node)
                node = int(tree[b, node])
            acc[b, :len(path)], n[b] = path[::-1], len(path)
        m.tree_accept_commit(table, seq, parents, to_dev(acc), to_dev(n), max_seq_len=max_len)
        table_np, lens, valid = oracle.tree_accept_commit(table_np, lens, tree, acc, n, max_len)
        assert valid.all()
        held_in.copy_(held_out)
        count_in.copy_(count_out)


def test_two_streams_at_once():
    """Two calls at a time with workspaces of their own, allocated inside the call for the stream that it runs on."""
    import torch
    import speculative_decode_mla_gb300 as m
    ps = [problem([4000 + 700 * i], 5, 6, 60 + i) for i in range(2)]
    dev = [(bf16_dev(p.q), to_dev(rows), to_dev(p.slot_table), to_dev(p.seq_lens), to_dev(p.tree_parent)) for p, rows, _ in ps]
    want = [m.verify_kv4(*d, max_seq_len=p.max_seq_len) for d, (p, _, _) in zip(dev, ps)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(m.verify_kv4(*dev[i], max_seq_len=ps[i][0].max_seq_len, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_two_graphs_replayed_in_turn():
    import torch
    import speculative_decode_mla_gb300 as m
    ps = [problem([900 + 700 * i], 3, 4, 70 + i) for i in range(2)]
    graphs, outs, wants = [], [], []
    for p, rows, bits in ps:
        dev = (bf16_dev(p.q), to_dev(rows), to_dev(p.slot_table), to_dev(p.seq_lens), to_dev(p.tree_parent))
        wants.append(m.verify_kv4(*dev, max_seq_len=p.max_seq_len))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.verify_kv4(*dev, max_seq_len=p.max_seq_len))
        graphs.append((g, dev))
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], wants[i][0]) and torch.equal(outs[i][1], wants[i][1])


@pytest.mark.slow
def test_slots_past_32_bit_byte_offsets():
    """Rows of a pool over 4 GiB: byte offsets past 2^32."""
    import torch
    import speculative_decode_mla_gb300 as m
    slots = (5 << 30) // 416
    pool = torch.zeros(slots, 416, dtype=torch.uint8, device="cuda")
    p, rows, bits = problem([400], 2, 3, 80)
    n = 402
    at = (slots - 1 - 7 * np.arange(n)).astype(np.int32)
    x = W.normal_bf16(81, n * 576).reshape(n, 576)
    m.kv4_append(pool, bf16_dev(x), to_dev(at))
    out = m.kv4_gather(pool, to_dev(at))
    values = oracle.kv4_bf16(oracle.kv4_quantise(x))
    assert np.array_equal(W.bf16_bits_to_f32(host_bf16(out)), W.bf16_bits_to_f32(values))
    table = np.zeros((1, n), np.int32)
    table[0] = at
    got = m.verify_kv4(bf16_dev(p.q), pool, to_dev(table), to_dev(p.seq_lens), to_dev(p.tree_parent), max_seq_len=400)
    want = oracle.verify(p.seq_lens, np.arange(n, dtype=np.int32)[None], p.tree_parent, p.q, values, num_heads=3, scale=W.SOFTMAX_SCALE)
    assert_close((got[0].float().cpu().numpy().reshape(-1, 512).astype(np.float64), got[1].cpu().numpy().reshape(-1).astype(np.float64)),
                 (want[0].reshape(-1, 512), want[1]), p.q, values)
