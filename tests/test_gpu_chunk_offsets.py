"""Chunk calls over offsets out of order or range: the sequences in front of the first such ones are right, and nothing else is
written, in the results or behind them."""
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import check, i32, offsets, tensor
from test_chunk_plan_host import good
from test_gpu_chunk import pool, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
KINDS = [(BF16, 64), (BF16, 128)]  # tcgen05

# offsets, Tq, query heads a key/value head, key/value heads, lengths
CALLS = [
    ([0, 68, 71, 195, 103, 128, 300], 300, 4, 2, [436, 2752, 56, 2755, 2210, 2195]),
    ([0, 1000, 200, 600], 600, 4, 2, [900] * 3),
    ([0, 971, 1679, 1080, 1145], 1679, 1, 1, [2500] * 4),
    ([0, 300, 200, 500], 500, 2, 2, [400, 400, 400]),
    ([0, 1, 2, 1, 3, 4], 4, 8, 2, [3000] * 5),
    ([-1, 3, 10], 10, 2, 2, [50, 500]),
    ([0, 40, 2 ** 31 - 1, 50], 50, 2, 2, [700, 500, 50]),
    ([0, 40, -2 ** 31, 50], 50, 2, 2, [700, 500, 50]),
    ([0, 20, 10 ** 6], 50, 2, 2, [700, 500]),
]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("call", range(len(CALLS)))
def test_bad_offsets(call, dtype, D):
    offs, Tq, G, Hk, lens = CALLS[call]
    n, H, guard = len(lens), G * Hk, 300
    cache, held = pool(lens, 64, Hk, D, dtype, 1)
    q = tensor((Tq, H, D), 5, dtype, DEV)
    a = moe.Attention(H, Hk, D, dtype)
    slots = i32(range(n), DEV)
    # what a call over good offsets of the same sizes leaves in the scratch memory
    a.chunk(q, cache, slots, i32(offsets([Tq // n] * n), DEV))
    assert a.device_status() == (moe.MOE_OK, 0)
    out = torch.full((Tq + guard, H, D), 5.0, dtype=dtype, device=DEV)
    lse = torch.full((Tq + guard, H), 5.0, dtype=F32, device=DEV)
    for _ in range(2):
        a.chunk(q, cache, slots, i32(offs, DEV), out=out[:Tq], lse=lse[:Tq])
        status, detail = a.device_status()
        bad = [i for i in range(n) if offs[i] < 0 or offs[i + 1] < offs[i] or offs[i + 1] > Tq]
        assert status == moe.MOE_ERR_DEVICE_CHECK and detail in bad
        seqs = good(offs, Tq)
        end = offs[seqs] if seqs else 0
        assert (out[end:] == 5).all() and (lse[end:] == 5).all()
        if seqs:
            ref = reference(q[:end], held, list(range(seqs)), offs[:seqs + 1], True, D ** -0.5)
            check(out[:end], lse[:end], ref, max(lens), D, dtype)
