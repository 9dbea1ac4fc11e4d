"""Workspaces of Attention on the GPU: what a larger one, a graph or a second thread does to them."""
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import i32, tensor
from test_gpu_attention import BF16, DEV, F32, make_cache

pytestmark = pytest.mark.gpu
BAD, OK = moe.MOE_ERR_DEVICE_CHECK, moe.MOE_OK


def setup(n=12, H=8, Hk=2, D=64, shared=64, dtype=BF16):
    c, _ = make_cache([shared + 5 + 11 * i for i in range(n)], shared, 16, Hk, D, dtype)
    return moe.Attention(H, Hk, D, dtype), c, tensor((n, H, D), 1, dtype, DEV)


@pytest.mark.parametrize("own_stream", [False, True])
def test_an_error_is_not_lost_when_the_workspace_grows(own_stream):
    a, c, q = setup()
    s = torch.cuda.Stream() if own_stream else None
    out = torch.empty_like(q)
    torch.cuda.synchronize()

    def call(slots):
        a.decode(q[:len(slots)], c, i32(slots, DEV), out=out[:len(slots)], stream=s)

    call([0, 99])
    for n in (3, 5, 12):
        call(list(range(n)))
    assert a.device_status() == (BAD, 1)
    assert a.device_status() == (OK, 0)


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_growing_batch_keeps_one_workspace(own_stream):
    a, c, q = setup(n=64, shared=32)
    s = torch.cuda.Stream() if own_stream else None
    want = a.decode(q, c, i32(range(64), DEV), shared_len=32)
    a = moe.Attention(8, 2, 64, BF16)
    out = torch.empty_like(q)
    slots = [i32(range(n), DEV) for n in range(65)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for n in range(1, 65):
        a.decode(q[:n], c, slots[n], shared_len=32, out=out[:n], stream=s)
    torch.cuda.synchronize()
    need = a._lib.moe_attention_workspace_bytes(64, 8, 64)
    assert torch.cuda.memory_allocated() - before <= 1.5 * need + 512
    assert torch.equal(out, want)
    assert a.device_status() == (OK, 0)
