"""How the wrappers make the tensors that they return: torch's short call for it where that is as it was known and nobody watches, else
torch's public one."""
import pytest
import torch

import speculative_decode_mla_gb300 as m


@pytest.fixture
def short_call(monkeypatch):
    """Puts a function in the place of torch's own short call."""
    def put(f):
        monkeypatch.setattr(torch._C._dynamo.guards, "_empty_strided_cuda", f, raising=False)
        m._empty_call.cache_clear()
    yield put
    m._empty_call.cache_clear()


@pytest.mark.parametrize("kind", ["other arguments", "something else", "a host tensor", "gone"])
def test_a_short_call_that_has_changed_is_not_used(short_call, kind):
    def other(size, device):
        raise AssertionError("called")
    short_call({"other arguments": other, "something else": lambda size, stride, dtype: 5,
                "a host tensor": lambda size, stride, dtype: torch.empty(size, dtype=dtype), "gone": None}[kind])
    like = torch.zeros(3)
    t = m._empty((4, 6), (6, 1), torch.bfloat16, like)
    assert t.shape == (4, 6) and t.stride() == (6, 1) and t.dtype is torch.bfloat16 and t.device == like.device


def wrappers():
    """(name, call) of each wrapper that makes tensors by the short call: small calls, which leave some rows unwritten."""
    d = dict(device="cuda")
    b = dict(dtype=torch.bfloat16, **d)
    i = dict(dtype=torch.int32, **d)
    rows, q = torch.ones(4, 576, **b), torch.ones(4, 2, 192, **b)
    pos, table = torch.tensor([0, -1, 1, -1], **i), torch.ones(2, 64, **d)
    k, kr = torch.ones(4, 2, 128, **b), torch.ones(4, 64, **b)
    pool4 = torch.zeros(8, 416, dtype=torch.uint8, **d)
    return {"rope_append": lambda: m.rope_append(None, rows, None, pos, table, q=q),
            "prompt_attn": lambda: m.prompt_attn(q, k, kr, k, torch.tensor([1, 3], **i), max_q_len=2),
            "kv4_gather": lambda: m.kv4_gather(pool4, torch.tensor([0, 3], **i))}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rope_append", "prompt_attn", "kv4_gather"])
def test_dispatch_modes_see_the_tensors(name):
    from torch.utils._python_dispatch import TorchDispatchMode
    call, seen = wrappers()[name], []

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    call()
    torch.cuda.synchronize()
    with Watch():
        call()
    assert any("empty" in f for f in seen), seen


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rope_append", "prompt_attn"])
def test_uninitialised_memory_is_filled_where_torch_is_told_to(name):
    call = wrappers()[name]
    call()
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True, warn_only=True)
    try:
        out, other = call()
    finally:
        torch.use_deterministic_algorithms(was)
    unwritten = [1, 3] if name == "rope_append" else [0, 3]
    assert torch.isnan(out[unwritten]).all() and torch.isnan(other[unwritten]).all()
