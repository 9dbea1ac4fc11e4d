"""Results that apply, append and chunk make themselves: as torch makes tensors, whatever way their memory comes."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import i32, tensor
from test_gpu_chunk import pool

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls(dtype):
    """Each call's results: of 5 tokens, the last two of no sequence; and all of apply's."""
    cache, _ = pool([53, 30], 16, 2, 64, dtype, 3)
    q, kv = tensor((5, 4, 64), 1, dtype, DEV), tensor((5, 2, 64), 2, dtype, DEV)
    rope, a = moe.Rotary(64), moe.Attention(4, 2, 64, dtype)
    slots, offs = i32([0, 1], DEV), i32([0, 2, 3], DEV)
    return {"apply": rope.apply(q, i32(range(5), DEV), kv)[0], "apply_k": rope.apply(q, i32(range(5), DEV), kv)[1],
            "append": cache.append(kv, kv, slots, offs, i32([51, 29], DEV), rope, q=q),
            "chunk": a.chunk(q, cache, slots, offs)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_new_memory_is_filled_under_deterministic_algorithms(dtype):
    plain = calls(dtype)
    torch.use_deterministic_algorithms(True)
    try:
        got = calls(dtype)
    finally:
        torch.use_deterministic_algorithms(False)
    for name, x in got.items():
        end = 5 if name.startswith("apply") else 3
        assert torch.equal(x[:end], plain[name][:end])
        assert torch.isnan(x[end:]).all()


def test_dispatch_modes_see_new_tensors():
    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            names.append(str(func))
            return func(*args, **(kwargs or {}))

    rope, q = moe.Rotary(64), tensor((5, 4, 64), 1, torch.bfloat16, DEV)
    pos, names = i32(range(5), DEV), []
    want = rope.apply(q, pos)
    with Seen():
        got = rope.apply(q, pos)
    assert any("empty_strided" in n for n in names) and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_the_short_way(dtype, monkeypatch):
    want = calls(dtype)
    monkeypatch.delattr(torch._C._dynamo.guards, "_empty_strided_cuda", raising=False)
    for name, x in calls(dtype).items():
        end = 5 if name.startswith("apply") else 3
        assert torch.equal(x[:end], want[name][:end])
        assert x.is_contiguous() and x.dtype is dtype and x.device == torch.device("cuda", 0)
