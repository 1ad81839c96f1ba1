"""The plan of attention over the 4-bit pool for calls of at most 16 query rows a sequence (no GPU)."""
import ctypes

import pytest

import speculative_decode_mla_gb300 as m
from speculative_decode_mla_gb300 import _build

SMS = 152


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return m.load_library()


def plan(lens, T=1, H=16, hint=None, room=None, splits=0, sms=SMS):
    room = max(lens) if room is None else room
    hint = sum(lens) + T * len(lens) if hint is None else hint
    return m.kv4_plan(m.make_desc(len(lens), T, H, 1 << 20, room + T, room, total_tokens_hint=hint, num_splits=splits), sms)


UNEVEN = [[131072] + [300] * (b - 1) for b in (16, 64, 256, 512, 700, 900, 1000, 2000)] + \
         [[16384] + [300] * (b - 1) for b in (64, 900, 4000)] + [[16000] * (b // 8) + [1000] * (b - b // 8) for b in (16, 64, 512, 1024)]


@pytest.mark.parametrize("lens", UNEVEN, ids=lambda l: f"{len(l)}x{max(l)}")
def test_a_long_sequence_among_short_ones_is_shared(lib, lens):
    """No CTA or pair of CTAs takes more positions of one sequence at a time than twice an even share of the whole batch, with
    a sequence's set-up counted as three tiles of 128 positions."""
    p = plan(lens)
    even = sum(n + 1 + 3 * 128 for n in lens) / (SMS // 2)
    assert p.chunk_tokens <= max(2 * even, 256), (p.kernel, p.chunk_tokens, even)
    assert p.kernel == 0


@pytest.mark.parametrize("b,n", [(16, 1000), (32, 8192), (64, 4096), (256, 1000), (1024, 300), (4096, 300), (4, 65536)])
def test_even_batches_take_the_kernel_for_few_rows(lib, b, n):
    for kw in ({}, dict(hint=0), dict(hint=0, room=2 * n)):
        assert plan([n] * b, **kw).kernel == 2
    assert plan([1 + n * i // b for i in range(b)]).kernel == (2 if b >= 16 else 0)   # lengths spread evenly from 1 on
    assert plan([n] * b, H=17).kernel == 0


@pytest.mark.parametrize("lens,kw", [([900] * 16, {}), ([900] * 16, dict(hint=0)), ([0] * 16, {}), ([1] * 16, {}), ([131072] * 16, {}),
                                     ([300] * 4096, {}), ([8192] * 1000, dict(hint=0)), ([5000] * 20, dict(splits=3)),
                                     ([5000] * 20, dict(splits=1000)), ([184320] * 60, dict(hint=0)), ([70000] * 4, {})])
@pytest.mark.parametrize("T,H", [(1, 16), (5, 3)])
def test_few_row_plans_cover_every_position(lib, lens, kw, T, H):
    p = plan(lens, T, H, **kw)
    assert p.kernel == 2 and p.rows_per_tile == 16 and p.row_tiles == 1
    n = max(lens) + T
    assert p.chunk_tokens % 64 == 0 and (p.num_splits - 1) * p.chunk_tokens < n <= p.num_splits * p.chunk_tokens
    assert p.ctas == len(lens) * p.num_splits
    assert p.workspace_bytes >= p.num_splits * len(lens) * T * H * (512 * 2 + 4)
