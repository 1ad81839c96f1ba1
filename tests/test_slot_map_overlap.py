"""mla_slot_map_build refuses arrays that overlap: a CTA sums the lengths of all sequences for itself, so an output that lies
over an input would let two CTAs read different numbers. The checks are the host's: refusals are tested without a GPU."""
import itertools

import pytest
import torch

import speculative_decode_mla_gb300 as m
from speculative_decode_mla_gb300 import _build

NAMES = ["seq", "new", "held", "B", "page", "pages", "free", "cap", "count", "block", "bstride", "slots", "sstride", "map", "mcap",
         "cu", "hout", "left", "debug", "status", "stream"]
B, PAGE, CAP, BSTRIDE, SSTRIDE, MCAP = 4, 16, 50, 8, 128, 64
SIZE = dict(seq=B, new=B, held=B, free=CAP, count=1, block=B * BSTRIDE, slots=B * SSTRIDE, map=MCAP, cu=B + 1, hout=B, left=1,
            status=1)                                         # int32 elements
WRITTEN = ["block", "slots", "map", "cu", "hout", "left", "status"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m.load_library()


def args(**kw):
    at = {n: (1 << 20) + 8192 * i for i, n in enumerate(SIZE)}
    a = dict(at, B=B, page=PAGE, pages=100, cap=CAP, bstride=BSTRIDE, sstride=SSTRIDE, mcap=MCAP, debug=1, stream=None)
    a.update(kw)
    return [a[n] for n in NAMES], a


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: only where no kernel can run")
@pytest.mark.parametrize("out,other", [(o, n) for o, n in itertools.product(WRITTEN, SIZE) if o != n])
def test_an_output_over_another_array_is_refused(lib, out, other):
    _, a = args()
    for shift in (0, 4 * (SIZE[other] - 1), -4 * (SIZE[out] - 1)):   # the same place, its last element, the output's last element
        assert lib.mla_slot_map_build(*args(**{out: a[other] + shift})[0]) == -1, shift


@pytest.mark.gpu
def test_arrays_back_to_back_in_one_allocation_are_taken():
    """Neighbours that touch do not overlap; seq_lens may serve as held_lens, and arrays of no elements lie anywhere."""
    import numpy as np
    import oracle
    rng = np.random.default_rng(3)
    seq, new = rng.integers(0, 50, B).astype(np.int32), rng.integers(1, 9, B).astype(np.int32)
    free, table = rng.permutation(CAP).astype(np.int32), np.full((B, SSTRIDE), -9, np.int32)
    block = np.tile(np.arange(50, 50 + BSTRIDE, dtype=np.int32), (B, 1))
    want = oracle.slot_map_build(seq, new, None, PAGE, 100, free, CAP, block, table, MCAP)
    buf = torch.zeros(sum(SIZE.values()), dtype=torch.int32, device="cuda")
    at, part = 0, {}
    for n in SIZE:
        part[n] = buf[at:at + SIZE[n]]
        at += SIZE[n]
    for n, v in dict(seq=seq, new=new, free=free, count=np.array([CAP], np.int32), block=block, slots=table).items():
        part[n].copy_(torch.from_numpy(v.reshape(-1)))
    tables = part["slots"].view(B, SSTRIDE), part["block"].view(B, BSTRIDE)
    kw = dict(page_size=PAGE, num_pages=100, held_lens=part["seq"], block_table=tables[1], cu_new=part["cu"], held_out=part["hout"],
              free_left=part["left"], debug=True, dev_status=part["status"])
    m.slot_map_build(part["seq"], part["new"], part["free"], part["count"], tables[0], slot_map=part["map"], **kw)
    for got, w in zip((tables[1], tables[0], part["map"], part["cu"], part["hout"]), want[:5]):
        assert np.array_equal(got.cpu().numpy(), w)
    assert part["left"].item() == want[5] and part["status"].item() == 0
    # a map of no elements inside cu_new, no free pages: nothing is granted, nothing is refused
    m.slot_map_build(part["seq"], part["new"], part["free"][:0], part["count"], tables[0], slot_map=part["cu"][1:1], **kw)
    assert part["status"].item() == m.CHECK_NO_PAGES
    with pytest.raises(m.MLAError):
        m.slot_map_build(part["seq"], part["new"], part["free"], part["count"], tables[0], slot_map=part["map"],
                         **dict(kw, cu_new=buf[SIZE["seq"] - 1:SIZE["seq"] + B]))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [False, True])
def test_pages_of_one_slot_in_one_table(bad):
    """One array as both tables; a page outside the pool leaves -1 in it."""
    import numpy as np
    import oracle
    seq, new = np.array([3, 0, 40], np.int32), np.array([4, 700, 1], np.int32)
    free, table = np.random.default_rng(5).permutation(800).astype(np.int32), np.full((3, 710), -9, np.int32)
    if bad:
        free[700] = 1 << 28
    want = oracle.slot_map_build(seq, new, None, 1, 800, free, 800, None, table, 720)
    dev = lambda x: torch.from_numpy(x.copy()).cuda()
    both = dev(table)
    got = m.slot_map_build(dev(seq), dev(new), dev(free), dev(np.array([800], np.int32)), both, page_size=1, num_pages=800,
                           map_capacity=720, block_table=both)
    assert np.array_equal(both.cpu().numpy(), want[1]) and np.array_equal(got[0].cpu().numpy(), want[2])
    assert (want[1] == -1).sum() == int(bad)
