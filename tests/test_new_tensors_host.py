"""Where results made by a call get their memory, with a torch that lacks the short way to the allocator or has it. Needs no GPU."""
from types import SimpleNamespace

import pytest

from sparse_mixture_experts_moe_gb300 import _lib


def fake(entry=True, deterministic=False, modes=0):
    calls = []
    t = SimpleNamespace(
        _C=SimpleNamespace(_len_torch_dispatch_stack=lambda: modes), are_deterministic_algorithms_enabled=lambda: deterministic,
        empty_strided=lambda shape, strides, dtype, device: calls.append(("dispatched", shape, strides, dtype, device)))
    if entry:
        t._C._dynamo = SimpleNamespace(guards=SimpleNamespace(
            _empty_strided_cuda=lambda shape, strides, dtype: calls.append(("entry", shape, strides, dtype, "cuda"))))
    return t, calls


@pytest.mark.parametrize("torch,way", [(fake(), "entry"), (fake(entry=False), "dispatched"), (fake(deterministic=True), "dispatched"),
                                       (fake(modes=1), "dispatched")])
def test_way(torch, way):
    _lib._allocator(torch[0])((2, 3, 8), (24, 8, 1), "bf16")
    assert torch[1] == [(way, (2, 3, 8), (24, 8, 1), "bf16", "cuda")]


def test_without_either_entry():
    torch, calls = fake()
    del torch._C._len_torch_dispatch_stack
    _lib._allocator(torch)((1,), (1,), "f32")
    assert calls[0][0] == "dispatched"
