"""Chunk calls over offsets out of order or range: they are recorded, what is computed is right, and nothing else is written, in
the results or behind them."""
import random

import numpy as np
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import check, i32, offsets, tensor
from test_chunk_plan_host import good
from test_gpu_chunk import pool, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
KINDS = [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128)]  # tcgen05, warp MMAs, CUDA cores

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


def run(offs, Tq, G, Hk, lens, dtype, D):
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
    valid = [i for i in range(n) if 0 <= offs[i] <= offs[i + 1] <= Tq]
    for _ in range(2):
        a.chunk(q, cache, slots, i32(offs, DEV), out=out[:Tq], lse=lse[:Tq])
        status, detail = a.device_status()
        if len(valid) < n:
            assert status == moe.MOE_ERR_DEVICE_CHECK and 0 <= detail < n and detail not in valid
        else:
            assert status == moe.MOE_OK
        left = ((out == 5).all(-1) & (lse == 5)).cpu().numpy()
        assert left[Tq:].all()
        claims = np.zeros(Tq, dtype=int)
        for i in valid:
            claims[offs[i]:offs[i + 1]] += 1
        assert left[:Tq][claims == 0].all()
        for i in valid:  # rows that one sequence alone has are right, or as they were
            rows = np.arange(offs[i], offs[i + 1])[claims[offs[i]:offs[i + 1]] == 1]
            if len(rows) == 0:
                continue
            ref = reference(q[offs[i]:offs[i + 1]], held, [i], [0, offs[i + 1] - offs[i]], True, D ** -0.5)
            ref = tuple(np.where(left[rows].reshape(left[rows].shape + (1,) * (x.ndim - 2)), 0 if k else 5.0, x[rows - offs[i]])
                        for k, x in enumerate(ref))
            ours = out[rows], torch.where(torch.tensor(left[rows], device=DEV), 0.0, lse[rows])
            check(*ours, ref, max(lens), D, dtype)
        if dtype == BF16 and D <= 128:  # the sequences end in front of the first bad offsets
            seqs = good(offs, Tq)
            mine = np.zeros(Tq, dtype=bool)
            mine[offs[0]:offs[seqs]] = seqs > 0
            assert (left[:Tq].all(-1) != mine).all() and (left[:Tq].any(-1) != mine).all()


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("call", range(len(CALLS)))
def test_bad_offsets(call, dtype, D):
    run(*CALLS[call], dtype, D)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("seed", range(12))
def test_random_bad_offsets(seed, dtype, D):
    r = random.Random(seed)
    n = r.choice([2, 3, 5, 9, 40])
    nq = [r.choice([0, 1, 2, 5, r.randint(1, 30), r.randint(1, 150 if n < 9 else 30)]) for _ in range(n)] + [1]
    lens = [r.choice([0, a, a + r.randint(0, 900)]) for a in nq]
    offs = offsets(nq)
    Tq = offs[-1] + r.choice([0, 3])
    for _ in range(r.choice([1, 1, 2, 4])):
        offs[r.randrange(len(offs))] = r.choice([r.randint(0, Tq), r.randint(0, Tq), r.randint(-40, Tq + 40), 2 ** 31 - 1,
                                                 -2 ** 31, -1, Tq + 1])
    run(offs, Tq, r.choice([1, 2, 7, 8]), r.choice([1, 2]), lens, dtype, D)
