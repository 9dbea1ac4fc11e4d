"""KVCache.append leaves what Rotary.apply and KVCache.write would, bit for bit, in the pages and in the queries."""
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import i32, offsets, tensor

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (80, 32), (256, 64), (24, 6), (200, 26), (64, 0)])
def test_append_is_apply_and_write(D, R, layout, norm, dtype):
    H, Hk, page, held, new = 6, 2, 16, [0, 5, 16, 100, 3], [7, 1, 40, 29, 0]
    n, T, offs = len(held), sum(new), offsets(new)
    x = tensor((T, H + 2 * Hk, D), D + R, dtype, DEV)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    wq, wk = (tensor((D,), s, dtype, DEV) if norm else None for s in (1, 2))
    rope = moe.Rotary(D, rotary_dim=R, layout=layout)
    slots, o, pos = i32([3, 0, 4, 1, 2], DEV), i32(offs, DEV), i32(held, DEV)
    caches = []
    for _ in range(2):
        c = moe.KVCache.create(1, 30, page, n, 256, Hk, D, dtype)
        c.k.fill_(7)
        c.v.fill_(7)
        c.resize(slots, i32([a + b for a, b in zip(held, new)], DEV))
        caches.append(c)
    got = caches[0].append(k, v, slots, o, pos, rope, q=q, q_weight=wq, k_weight=wk)
    at = i32([p for a, b in zip(held, new) for p in range(a, a + b)], DEV)
    want, turned = rope.apply(q, at, k, q_weight=wq, k_weight=wk)
    caches[1].write(turned, v, slots, o, pos)
    assert torch.equal(caches[0].table, caches[1].table)
    assert torch.equal(got, want) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    assert all(c.device_status() == (moe.MOE_OK, 0) for c in caches)
