"""A pair of CTAs that works on one sequence for longer than a wait inside the kernel may take, and has others after it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.slow
def test_a_segment_longer_than_the_limit_of_a_wait():
    """166 million positions in one part, about 2.3 s of one pair, then two short sequences by the same pair. One position of each
    sequence lies 40 above the others in score, which all share a slot: 2^28 e^-40 is below 2^-29, so its values are the output and
    its score is the lse, to ten roundings of a number below 2^6."""
    import torch
    import oracle
    import speculative_decode_mla_gb300 as m
    lens, room = [128 * 1_300_000 - 1, 300, 20], 128 * 1_310_000
    x = np.zeros((2, 576), np.float32)
    x[:, :512] = np.random.default_rng(4).choice([-1.0, 1.0], (2, 512))
    x[1, 512] = 64.0
    rows = oracle.kv4_quantise((x.view(np.uint32) >> 16).astype(np.uint16))
    values = oracle.kv4_values(rows)
    q = torch.zeros(3, 1, 576, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 512] = torch.tensor([9.0, 9.5, 10.0])
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.zeros(3, room + 1, **i32)
    table[torch.arange(3), torch.tensor([100_000_000, 299, 20])] = 1
    st = torch.zeros(1, **i32)
    out, lse = m.verify_kv4(q, torch.from_numpy(rows).cuda(), table, torch.tensor(lens, **i32), torch.full((3, 1), -1, **i32),
                            max_seq_len=room, num_splits=1, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert np.array_equal(out.float().cpu().numpy(), np.tile(values[None, 1:, :512], (3, 1, 1)))
    assert np.abs(lse.cpu().numpy()[:, 0] - np.array([9.0, 9.5, 10.0]) * 64 * m.DEFAULT_SCALE).max() <= 10 * 2.0 ** -24 * 2 ** 6
