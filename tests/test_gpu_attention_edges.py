"""Attention over the paged cache and over packed prompts where calls are unusual: batches of several slices, tables
and lengths that do not hold what the call says, non-finite values, scales at the ends of their range."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import attend64, check, f64, i32, offsets, prompt_reference, tensor
from test_gpu_attention import BF16, DEV, F32, decode_reference, make_cache

pytestmark = pytest.mark.gpu
BAD = moe.MOE_ERR_DEVICE_CHECK


def trim(c, lens):
    """Table entries past the slots' lengths become -1, as the cache's calls leave them."""
    for i, a in enumerate(lens):
        c.table[i, -(-a // c.page_size):] = -1


def decode(c, H, D, dtype, slots, shared, seed=5, scale=None):
    """(out, lse, q, (status, detail)) of one decode call; out and lse hold NaN before it."""
    q = tensor((len(slots), H, D), seed, dtype, DEV)
    a = moe.Attention(H, c.kv_heads, D, dtype, scale=scale)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    a.decode(q, c, i32(slots, DEV), shared_len=shared, out=out, lse=lse)
    return out, lse, q, a.device_status()


def right(out, lse, q, c, rows, lens, at, D, dtype):
    """Rows `at` of a decode call whose row i attends slot i."""
    ref = decode_reference(q[at], c, [rows[i] for i in at], [lens[i] for i in at], 0, D ** -0.5)
    check(out[at], lse[at], ref, max(lens), D, dtype)


# ---------------------------------------------------------------------------------------- batches of several slices

@pytest.mark.parametrize("short", [0, 5, 16])
def test_decode_slices_share_the_calls_first_slot(short):
    """2048 sequences are one slice of a call: the prefix's pages are those of the call's first slot, also where a
    later slice begins with a slot that does not hold all of it."""
    n, shared = 2100, 48
    lens = [shared + 1 + i % 20 for i in range(n)]
    lens[2048] = lens[2060] = short
    c, rows = make_cache(lens, shared, 16, 1, 32, BF16)
    trim(c, lens)
    out, lse, q, st = decode(c, 2, 32, BF16, range(n), shared)
    assert st == (moe.MOE_OK, 0)
    right(out, lse, q, c, rows, lens, list(range(n)), 32, BF16)


@pytest.mark.parametrize("bad", [-1, 5000])
def test_decode_slice_that_begins_with_a_bad_slot(bad):
    n, shared = 2060, 32
    lens = [shared + 1 + i % 20 for i in range(n)]
    c, rows = make_cache(lens, shared, 16, 1, 32, BF16)
    c.table[0] = -1  # a slot that the call does not name
    c.lens[0] = 0
    slots = [1 + i % (n - 1) for i in range(n)]
    slots[2048] = bad
    out, lse, q, st = decode(c, 2, 32, BF16, slots, shared)
    assert st == (BAD, 2048)
    assert (out[2048] == 0).all()
    at = [i for i in range(n) if i != 2048]
    ref = decode_reference(q[at], c, [rows[slots[i]] for i in at], [lens[slots[i]] for i in at], 0, 32 ** -0.5)
    check(out[at], lse[at], ref, max(lens), 32, BF16)
