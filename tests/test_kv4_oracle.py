"""Pins of the 4-bit row format's and the slot map's definitions, and the new entry points' refusals (no GPU)."""
import ctypes

import numpy as np
import pytest

import oracle
import speculative_decode_mla_gb300 as m
from speculative_decode_mla_gb300 import _build
from speculative_decode_mla_gb300 import workloads as W


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m.load_library()


def rows_of(x):
    """float32 [n, 576] as bf16 bits."""
    return W.f32_to_bf16_bits(np.asarray(x, dtype=np.float32)).reshape(-1, 576)


def test_e4m3_and_e2m1_tables_match_torch():
    import torch
    b = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(b.view(torch.float8_e4m3fn).double().numpy(), oracle.E4M3)
    assert oracle.E4M3[126] == 448 and oracle.E4M3[1] == 2.0 ** -9


def test_quantise_known_blocks():
    x = np.zeros((4, 576), dtype=np.float32)
    x[0, :16] = [6, 4, 3, 2, 1.5, 1, 0.5, 0, -6, -4, -3, -2, -1.5, -1, -0.5, 0]   # scale 1: every code exactly
    x[0, 16:32] = 12 * np.array([1, 0.25 / 6, 0.75 / 6, 1.25 / 6, 1.75 / 6, 2.5 / 6, 3.5 / 6, 5 / 6] * 2)  # ties, scale 2
    x[1, :16] = 6 * 2.0 ** -11                                                    # the scale rounds to 0
    x[2, :16] = 1e6                                                               # saturates
    x[3, 5] = np.inf
    x[3, 20] = np.nan
    x[:, 512:] = np.arange(64) - 31.5
    bits = rows_of(x)
    v = oracle.kv4_values(oracle.kv4_quantise(bits))
    assert np.array_equal(v[0, :16], x[0, :16])
    assert np.array_equal(v[0, 16:24], [12, 0, 2, 2, 4, 4, 8, 8])                 # ties go to the even code
    assert (v[1, :512] == 0).all() and (v[2, :16] == 2688).all()
    assert np.isnan(v[3, :32]).all() and (v[3, 32:512] == 0).all()
    assert np.array_equal(v[:, 512:], x[:, 512:])


def test_quantise_is_off_by_half_a_step():
    """A code is the nearest of e2m1's values (steps of 0.5, 1 and 2 up to 2, 4 and 6), so a dim is off by at most half of its step x scale
    plus what the scale's rounding (at most 2^-4) puts above 6."""
    bits = W.normal_bf16(5, 64 * 576).reshape(64, 576)
    x = oracle._bf16_values(bits)[:, :512].reshape(64, 32, 16)
    rows = oracle.kv4_quantise(bits)
    v = oracle.kv4_values(rows)[:, :512].reshape(64, 32, 16)
    s = oracle.E4M3[rows[:, 256:288]][:, :, None]
    assert (np.abs(s * 6 / np.abs(x).max(axis=2, keepdims=True) - 1) <= 2.0 ** -4).all()
    y = np.abs(x) / s
    half = np.where(y <= 2, 0.25, np.where(y <= 4, 0.5, 1.0))
    assert (np.abs(x - v) <= half * s).all()


def test_values_are_bf16_numbers_for_every_code_and_scale():
    rows = np.zeros((256, 416), dtype=np.uint8)
    rows[:, :256] = np.arange(256)[None, :]
    rows[:, 256:288] = np.arange(256)[:, None]
    oracle.kv4_bf16(rows)   # asserts


def test_slot_map_small_by_hand():
    block = np.zeros((2, 4), dtype=np.int32)
    block[0, 0] = 9
    table = np.full((2, 8), -5, dtype=np.int32)
    table[0, :3] = [18, 19, 99]
    # pages of two slots; sequence 0 holds 3 positions, of which 2 are prefix, and wants 3 from position 2 on
    got = oracle.slot_map_build([2, 0], [3, 1], [3, 0], 2, 50, np.array([7, 8, 3, 4], np.int32), 4, block, table, 6)
    block2, table2, slot_map, cu, held, left, bits = got
    assert block2[0].tolist() == [9, 0, 4, 0] and block2[1].tolist() == [3, 0, 0, 0]
    assert table2[0].tolist() == [18, 19, 99, 1, 8, -5, -5, -5] and table2[1, 0] == 6
    assert slot_map.tolist() == [99, 1, 8, 6, -1, -1] and cu.tolist() == [0, 3, 4] and held.tolist() == [5, 1]
    assert left == 2 and bits == set()


# ------------------------------------------------------------------------------------------ refusals

FAKE = 1 << 20


def test_append_and_gather_refuse(lib):
    f = lib.mla_kv4_append
    ok = [FAKE, 10, FAKE, 576, FAKE, 4, 0, None, None]
    bad = [(0, None), (0, FAKE + 16), (1, 0), (1, 1 << 31), (2, None), (2, FAKE + 2), (3, 575), (3, 580), (4, None), (4, FAKE + 2),
           (5, -1), (6, 1)]
    for i, v in bad:
        args = list(ok)
        args[i] = v
        assert f(*args) == -1, (i, v)
    assert f(None, 10, None, 576, None, 0, 0, None, None) == 0        # no rows: nothing to do
    g = lib.mla_kv4_gather
    ok = [FAKE, 10, FAKE, 4, FAKE, 0, None, None]
    for i, v in [(0, None), (0, FAKE + 16), (1, 0), (2, None), (2, FAKE + 1), (3, -2), (4, None), (4, FAKE + 8), (5, 1)]:
        args = list(ok)
        args[i] = v
        assert g(*args) == -1, (i, v)
    assert g(None, 10, None, 0, None, 0, None, None) == 0


def test_slot_map_refuses(lib):
    f = lib.mla_slot_map_build
    names = ["seq", "new", "held", "B", "page", "pages", "free", "cap", "count", "block", "bstride", "slots", "sstride", "map",
             "mcap", "cu", "hout", "left", "debug", "status", "stream"]
    p = lambda k: FAKE + 4096 * k
    ok = dict(seq=p(0), new=p(1), held=p(2), B=4, page=16, pages=100, free=p(3), cap=50, count=p(4), block=p(5), bstride=8,
              slots=p(6), sstride=128, map=p(7), mcap=64, cu=p(8), hout=p(9), left=p(10), debug=0, status=None, stream=None)
    bad = [dict(seq=None), dict(new=None), dict(count=None), dict(slots=None), dict(cu=None), dict(hout=None), dict(left=None),
           dict(free=None), dict(map=None), dict(B=0), dict(page=0), dict(pages=0), dict(pages=1 << 30), dict(cap=-1), dict(sstride=0),
           dict(mcap=-1), dict(mcap=1 << 31), dict(block=None), dict(bstride=0), dict(hout=p(2)), dict(hout=p(0)), dict(hout=p(1)),
           dict(left=p(4)), dict(debug=1), dict(map=p(7) + 2), dict(held=p(2) + 1)]
    for b in bad:
        assert f(*[{**ok, **b}[n] for n in names]) == -1, b
    assert f(*[{**ok, "B": 8193}[n] for n in names]) == -2


def desc(**kw):
    base = dict(num_seqs=1, num_nodes=16, num_heads=8, num_slots=131072, slot_table_stride=65552, max_seq_len=65536)
    base.update(kw)
    return m.make_desc(base.pop("num_seqs"), base.pop("num_nodes"), base.pop("num_heads"), base.pop("num_slots"),
                       base.pop("slot_table_stride"), base.pop("max_seq_len"), **base)


def test_verify_kv4_refuses(lib):
    f = lib.mla_verify_attn_kv4
    d = desc()
    ok = [FAKE] * 10 + [1 << 40, None, None]   # q pool table lens sizes parent out lse (workspace)
    ok = [FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 40, None, None]
    for i in (0, 1, 2, 3, 5, 6, 7, 8):
        for v in (None, FAKE + 2):
            args = list(ok)
            args[i] = v
            assert f(ctypes.byref(d), *args) == -1, (i, v)
    args = list(ok)
    args[1] = FAKE + 16                         # the pool's alignment is 32
    assert f(ctypes.byref(d), *args) == -1
    args = list(ok)
    args[4] = FAKE + 2
    assert f(ctypes.byref(d), *args) == -1
    args = list(ok)
    args[8] = FAKE + 128                        # the workspace's alignment is 256
    assert f(ctypes.byref(d), *args) == -1
    assert f(ctypes.byref(desc(flags=m.MLA_FLAG_DEBUG_CHECKS)), *ok) == -1
    assert f(ctypes.byref(desc(num_nodes=65)), *ok) == -2
    assert f(None, *ok) == -1


@pytest.mark.parametrize("bad", [dict(num_nodes=0), dict(num_nodes=65), dict(num_heads=0), dict(num_seqs=0),
                                 dict(slot_table_stride=100), dict(num_slots=0), dict(max_seq_len=-1),
                                 dict(softmax_scale=float("inf")), dict(out_dtype=2), dict(flags=1 << 9),
                                 dict(num_splits=-1), dict(max_seq_len=2 ** 31 - 70, slot_table_stride=2 ** 31 - 1),
                                 dict(num_seqs=2000, max_seq_len=2 ** 28, slot_table_stride=2 ** 29, num_heads=64)])
def test_kv4_plan_refuses(lib, bad):
    assert lib.mla_verify_kv4_plan(ctypes.byref(desc(**bad)), 152, ctypes.byref(m.Plan())) in (-1, -2)


@pytest.mark.parametrize("kw", [dict(), dict(max_seq_len=0), dict(num_heads=1, num_nodes=1), dict(num_heads=64, num_nodes=64, slot_table_stride=65600),
                                dict(num_seqs=32, total_tokens_hint=200000), dict(num_seqs=100), dict(num_splits=7),
                                dict(flags=m.MLA_FLAG_SIMT), dict(num_seqs=3, total_tokens_hint=1)])
def test_kv4_plan_covers_every_position(lib, kw):
    d = desc(**kw)
    p = m.kv4_plan(d, 152)
    n = d.max_seq_len + d.num_nodes
    # a row tile's positions may begin inside a share of chunk_tokens; a single one is shared by all 76 pairs of SMs
    cover = -(-n // p.chunk_tokens)
    most = cover if p.kernel else max(cover + 2, min(-(-n // 128), 76))
    assert p.chunk_tokens % 64 == 0 and cover <= p.num_splits <= most
    assert p.row_tiles * p.rows_per_tile >= d.num_nodes * d.num_heads
    rows = d.num_seqs * d.num_nodes * d.num_heads
    assert p.workspace_bytes >= p.num_splits * rows * (512 * 2 + 4)
