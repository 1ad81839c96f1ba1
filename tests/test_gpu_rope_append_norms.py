"""mla_rope_append as a layer runs it, the latent rows normalised on their way into the 4-bit pool, over more rows than one block has; and
heads of sizes that leave lanes idle. The checks and tolerances are those of test_gpu_rope_append.py."""
import pytest

import test_gpu_rope_append as rope

pytestmark = pytest.mark.gpu
built = rope.built


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("n,heads,dim,width,fmt", [(4099, 0, 64, 2112, "kv4"), (777, 64, 64, 2112, "kv4"), (1500, 5, 72, 576, "bf16"),
                                                   (900, 3, 136, 584, "kv4"), (300, 2, 168, 576, "none")])
def test_norms_over_many_rows(n, heads, dim, width, fmt, halves):
    rope.test_rows_heads_and_pool(n, heads, dim, width, fmt, True, halves)


@pytest.mark.parametrize("fmt", ["bf16", "kv4"])
def test_rows_of_zeros_and_of_one_value(fmt):
    """eps alone under the root; and rows whose blocks of the 4-bit row are all zeros but one."""
    import numpy as np
    import torch
    import oracle
    import speculative_decode_mla_gb300 as m
    rng = np.random.default_rng(3)
    n = 70
    x = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(1, n), 8 * torch.arange(1, n) % 576] = rope.bf16_of(rng, n - 1)
    pos, table, slots = rope.to_dev(np.arange(n, dtype=np.int32)), rope.to_dev(rope.cos_sin(rng, n)), rope.to_dev(rng.permutation(n).astype(np.int32))
    w = rope.bf16_of(rng, 512)
    pool = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda") if fmt == "bf16" else torch.zeros(n, 416, dtype=torch.uint8, device="cuda")
    rows, _ = m.rope_append(pool, x, slots, pos, table, weight=w, eps=1e-6)
    rope.check(rope.values(x), None, rope.values(table), rope.values(w), None, 1e-6, False, rows, None)
    assert (rows[0] == 0).all()
    want = rows if fmt == "bf16" else rope.to_dev(oracle.kv4_quantise(rope.host_bits(rows)))
    assert torch.equal(pool[slots.long()].view(torch.uint8), want.view(torch.uint8))
