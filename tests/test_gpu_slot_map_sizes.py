"""mla_slot_map_build at the numbers of sequences where its shared memory passes the default limit, in a process of its own:
a call with more sequences earlier in a process hides a limit that was not raised."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = """
import numpy as np, torch
import oracle
import speculative_decode_mla_gb300 as m
for B in (6111, 6112, 6128, 6143, 6144, 8192):
    rng = np.random.default_rng(B)
    seq, new = rng.integers(0, 4, B).astype(np.int32), rng.integers(0, 4, B).astype(np.int32)
    slots = rng.permutation(8 * B).astype(np.int32)
    table = slots[:8 * B].reshape(B, 8)[:, :7].copy()
    free = slots[::-1][:4 * B].copy()
    cap = int(new.sum()) + 5
    dev = lambda x: torch.from_numpy(x.copy()).cuda()
    table_d = dev(table)
    got = m.slot_map_build(dev(seq), dev(new), dev(free), dev(np.array([len(free)], np.int32)), table_d, page_size=1,
                           num_pages=8 * B, map_capacity=cap)
    want = oracle.slot_map_build(seq, new, None, 1, 8 * B, free, len(free), None, table, cap)
    for g, w in zip(got, want[2:5]):
        assert np.array_equal(g.cpu().numpy(), w), B
    assert got[3].item() == want[5] and np.array_equal(table_d.cpu().numpy(), want[1]), B
    print("ok", B, flush=True)
"""


def test_slot_map_takes_every_number_of_sequences_in_a_fresh_process():
    from speculative_decode_mla_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT}, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, f"after {r.stdout.split(chr(10))[-2:]}: {r.stderr[-800:]}"
