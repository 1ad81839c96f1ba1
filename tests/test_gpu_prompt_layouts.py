"""Places and layouts of what mla_prompt_attn and mla_rope_append read and write (include/mla_prompt.h): results are the same bits wherever
the tensors lie, as far as the kernels promise to take them."""
import numpy as np
import pytest

from _helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decode_mla_gb300 import _build
    _build.build()


def normal(rng, *shape):
    import torch
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(torch.bfloat16).cuda()


def ints(v):
    return to_dev(np.asarray(v, np.int32))


def problem(m, n, heads, seed=1):
    rng = np.random.default_rng(seed)
    ends = lambda v: ints(np.concatenate([[0], np.cumsum(v)]))
    kv, rows = normal(rng, sum(n), heads, 256), normal(rng, sum(n), 576)
    return dict(q=normal(rng, sum(m), heads, 192), k_nope=kv[..., :128], k_rope=rows[:, 512:], v=kv[..., 128:], cu_q=ends(m), cu_k=ends(n),
                max_q_len=max(m), max_k_len=max(n))


def same(a, b):
    import torch
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,ctas", [([70, 9], [70, 300], 0), ([70, 9], [70, 300], 3), ([300, 140], [300, 520], 0), ([300, 140], [300, 520], 5)])
def test_outputs_aligned_to_16_bytes_and_no_more(m, n, ctas, f32, flags):
    import torch
    import speculative_decode_mla_gb300 as lib
    p = problem(m, n, 2)
    kw = dict(num_ctas=ctas, flags=lib.MLA_FLAG_SIMT if flags == "simt" else 0, out_dtype=lib.MLA_DTYPE_F32 if f32 else lib.MLA_DTYPE_BF16)
    want = lib.prompt_attn(**p, **kw)
    size, at = want[0].numel(), 4 if f32 else 8
    room = torch.full((size + 2 * at,), 7.0, dtype=want[0].dtype, device="cuda")
    lse_room = torch.full((want[1].numel() + 2,), 7.0, device="cuda")
    out, lse = room[at:at + size].view(want[0].shape), lse_room[1:-1].view(want[1].shape)
    assert room.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 16
    assert same(lib.prompt_attn(**p, **kw, out=out, lse=lse), want)
    assert (room[:at] == 7).all() and (room[at + size:] == 7).all() and lse_room[0] == 7 and lse_room[-1] == 7


@pytest.mark.parametrize("flags", ["simt", "tc"])
@pytest.mark.parametrize("m,ctas", [(200, 0), (200, 3), (90, 0), (90, 4)])
def test_prompt_offsets_past_31_bits(m, ctas, flags):
    """Token strides of 2^24 elements: the last rows lie 3.3 * 10^9 elements behind the first."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p, n, far = problem([m], [200], 2), 200, 1 << 24
    room = torch.empty(n * far, dtype=torch.bfloat16, device="cuda")
    view = lambda t, at: room.as_strided(t.shape, (far, 4096, 1) if t.dim() == 3 else (far, 1), at).copy_(t)
    wide = {**p, "q": view(p["q"], 0), "k_nope": view(p["k_nope"], 1 << 20), "v": view(p["v"], 1 << 21), "k_rope": view(p["k_rope"], 1 << 22)}
    kw = dict(num_ctas=ctas, flags=lib.MLA_FLAG_SIMT if flags == "simt" else 0)
    assert same(lib.prompt_attn(**wide, **kw), lib.prompt_attn(**p, **kw))


def test_graphs_that_share_a_workspace():
    """Captured calls of one workspace, replayed in turn on one stream, with anything left in it before each."""
    import torch
    import speculative_decode_mla_gb300 as lib
    calls = [(problem([40, 130], [900, 1300], 2, seed=3), dict(num_ctas=9)), (problem([300], [1500], 4, seed=4), dict(num_ctas=20)),
             (problem([17] * 30, [200] * 30, 2, seed=5), dict(num_ctas=0))]
    want = [lib.prompt_attn(**p, **kw) for p, kw in calls]
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for p, kw in calls:
        out, lse = torch.empty_like(want[len(got)][0]), torch.empty_like(want[len(got)][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(lib.prompt_attn(**p, **kw, out=out, lse=lse, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 2, 1, 0, 2, 2):
        ws.fill_(255)
        got[i][0].zero_()
        graphs[i].replay()
        graphs[(i + 1) % 3].replay()
        torch.cuda.synchronize()
        assert same(got[i], want[i]) and same(got[(i + 1) % 3], want[(i + 1) % 3])


@pytest.mark.parametrize("fmt", ["bf16", "kv4"])
def test_rope_offsets_past_31_bits(fmt):
    """Rows and heads with token strides of 2^24 elements, slots behind the pool's first 2^31 elements (bytes of the 4-bit pool)."""
    import torch
    import speculative_decode_mla_gb300 as lib
    rng = np.random.default_rng(2)
    n, heads, far = 150, 3, 1 << 24
    rows, q = normal(rng, n, 576), normal(rng, n, heads, 192)
    a = rng.normal(size=(n, 32))
    table, pos = to_dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)), ints(np.arange(n))
    slots = 4_000_000 if fmt == "bf16" else 5_500_000
    at = ints(slots - 1 - 2 * np.arange(n))
    pool = torch.zeros(slots, 576, dtype=torch.bfloat16, device="cuda") if fmt == "bf16" else torch.zeros(slots, 416, dtype=torch.uint8, device="cuda")
    small = torch.zeros(2 * n, *pool.shape[1:], dtype=pool.dtype, device="cuda")
    w, qw = normal(rng, 512), normal(rng, 192)
    want = lib.rope_append(small, rows, ints(2 * n - 1 - 2 * np.arange(n)), pos, table, weight=w, q=q, q_weight=qw)
    room = torch.empty(n * far, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((n, 576), (far, 1), 0).copy_(rows)
    y = room.as_strided((n, heads, 192), (far, 1 << 12, 1), 1 << 20).copy_(q)
    z = room.as_strided((n, heads, 192), (far, 1 << 12, 1), 1 << 21)
    got = lib.rope_append(pool, x, at, pos, table, weight=w, q=y, q_weight=qw, q_out=z)
    assert same(got, want) and torch.equal(pool[-2 * n:], small) and not pool[:-2 * n].any()


def test_rows_out_and_heads_in_place_over_their_inputs():
    """rows_out on rows (stride 576) and q_out on q: every element is read before it is written."""
    import torch
    import speculative_decode_mla_gb300 as lib
    rng = np.random.default_rng(6)
    n = 1000
    rows, q = normal(rng, n, 576), normal(rng, n, 5, 72)
    a = rng.normal(size=(n, 32))
    table, pos = to_dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)), ints(rng.permutation(n))
    w, qw = normal(rng, 512), normal(rng, 72)
    want = lib.rope_append(None, rows, None, pos, table, weight=w, q=q, q_weight=qw, halves=True)
    r, h = rows.clone(), q.clone()
    lib.rope_append(None, r, None, pos, table, weight=w, q=h, q_weight=qw, halves=True, rows_out=r, q_out=h)
    assert same((r, h), want)


@pytest.mark.parametrize("ctas", [0, 3, 152])
def test_ends_that_fall_are_reported_and_stay_in_bounds(ctas):
    """Ends that fall again and again give more units than the rows of q can make: what there is no room for is left out."""
    import torch
    import speculative_decode_mla_gb300 as lib
    p = problem([1000], [1000], 2, seed=7)
    want = lib.prompt_attn(**p, num_ctas=ctas)
    bad = {**p, "cu_q": ints([0, 1000] * 5), "cu_k": ints([0, 1000] * 5)}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.prompt_attn(**bad, num_ctas=ctas)
    with pytest.raises(lib.MLAError):
        lib.prompt_attn(**bad, num_ctas=ctas, flags=lib.MLA_FLAG_DEBUG_CHECKS, dev_status=status)
    assert int(status) == lib.CHECK_BAD_LENGTH
    assert same(lib.prompt_attn(**p, num_ctas=ctas), want)
