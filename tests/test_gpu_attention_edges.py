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


# --------------------------------------------------------------------------- slots that do not share what the call says

def other_page(c, slot, column):
    """The slot's page of that column becomes another valid page."""
    c.table[slot, column] = (c.table[slot, column] + 1) % c.n_pages


@pytest.mark.parametrize("n,pages,row", [(64, 512, 63), (64, 512, 5), (64, 512, 32), (3, 700, 2), (70, 9, 40)])
@pytest.mark.parametrize("H,Hk,D", [(8, 1, 64), (16, 8, 128), (12, 2, 64)])
def test_decode_other_pages_are_recorded(n, pages, row, H, Hk, D):
    """Wherever they lie, and however few positions the sequences have of their own."""
    lens = [16 * pages + (i == 1) for i in range(n)]
    c, rows = make_cache(lens, 16 * pages, 16, Hk, D, BF16)
    for column in (0, pages // 2, pages - 1):
        was = c.table.clone()
        other_page(c, row, column)
        out, lse, q, st = decode(c, H, D, BF16, range(n), 16 * pages)
        assert st == (BAD, row), column
        c.table.copy_(was)
        if column == 0:  # the other rows are right
            right(out, lse, q, c, rows, lens, [i for i in (1, n - 1) if i != row], D, BF16)
    assert decode(c, H, D, BF16, range(n), 16 * pages)[3] == (moe.MOE_OK, 0)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 256), (BF16, 136), (BF16, 256), (BF16, 64)])
@pytest.mark.parametrize("n", [2, 3, 5, 6, 9])
def test_decode_other_pages_are_recorded_for_few_sequences(n, dtype, D):
    """Also where each sequence reads the shared positions for itself."""
    lens = [64] * n
    c, rows = make_cache(lens, 64, 16, 2, D, dtype)
    for row, column in ((1, 0), (n - 1, 3)):
        was = c.table.clone()
        other_page(c, row, column)
        assert decode(c, 4, D, dtype, range(n), 64)[3] == (BAD, row)
        c.table.copy_(was)


@pytest.mark.parametrize("n,dtype,D", [(7, BF16, 64), (2, BF16, 64), (7, F32, 64), (2, F32, 64), (7, BF16, 256), (2, BF16, 256)])
def test_decode_a_first_slot_without_the_prefix_is_recorded(n, dtype, D):
    lens = [40] + [70] * (n - 1)
    c, rows = make_cache(lens, 64, 16, 2, D, dtype)
    trim(c, lens)
    assert decode(c, 4, D, dtype, range(n), 64)[3] == (BAD, 0)


@pytest.mark.parametrize("value", [-1, 1 << 20])
@pytest.mark.parametrize("n,dtype,D", [(7, BF16, 64), (2, BF16, 64), (7, F32, 64), (2, F32, 64), (7, BF16, 256), (2, BF16, 256)])
def test_decode_shared_pages_out_of_range_are_recorded(n, dtype, D, value):
    lens = [64] * n
    c, rows = make_cache(lens, 64, 16, 2, D, dtype)
    c.table[:, 2] = value  # the same in every slot
    st, row = decode(c, 4, D, dtype, range(n), 64)[3]
    assert st == BAD and 0 <= row < n


# ---------------------------------------------------------------------------------------------- lengths out of range

@pytest.mark.parametrize("length", [-5, 1 << 30, None])
@pytest.mark.parametrize("shared", [0, 32])
@pytest.mark.parametrize("n,dtype,D", [(7, BF16, 64), (2, BF16, 128), (7, F32, 64), (2, F32, 64), (3, F32, 256), (7, BF16, 256),
                                       (2, BF16, 256)])
def test_decode_bad_lengths_are_recorded(n, dtype, D, shared, length):
    """On every path a length outside [0, width * page size] is an error, and its row one that sees nothing."""
    lens = [60] * n
    c, rows = make_cache(lens, 32, 16, 2, D, dtype)
    c.lens[1] = c.width * 16 + 1 if length is None else length
    out, lse, q, st = decode(c, 4, D, dtype, range(n), shared)
    assert st == (BAD, 1)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    right(out, lse, q, c, rows, lens, [i for i in range(n) if i != 1], D, dtype)


# ------------------------------------------------------------------------------------------------- non-finite values

@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("page,pages", [(16, 9), (32, 1), (64, 3), (256, 1)])
def test_decode_infinite_shared_value_stays_infinite(page, pages, value):
    """An infinite value at the end of the shared positions, which are no whole number of blocks: rows that see it get
    that infinity, not a NaN."""
    shared, n, D = page * pages, 5, 64
    lens = [shared + i for i in range(n)]
    c, rows = make_cache(lens, shared, page, 2, D, BF16)
    for at in (shared - 1, shared - page):
        c.v[0, rows[0][at // page], 1, at % page, 5] = value
    out, lse, q, st = decode(c, 8, D, BF16, range(n), shared)
    assert st == (moe.MOE_OK, 0)
    assert (out[:, 4:, 5] == value).all()
    assert torch.isfinite(out[:, :4]).all() and torch.isfinite(out[:, 4:, 6:]).all()


@pytest.mark.parametrize("D", [64, 128, 200, 256])
@pytest.mark.parametrize("nq,nk", [([700], [700]), ([40, 300], [900, 300]), ([9, 2], [2500, 64])])
def test_prompt_values_that_are_not_finite_in_many_columns(nq, nk, D):
    """Infinities and NaN at many positions and columns: what a row does not see leaves its columns as they are, and what it
    does see makes them what the formula says."""
    H, Hk = 4, 2
    q, k, v = (tensor((sum(x), h, D), s, BF16, DEV) for x, h, s in ((nq, H, 1), (nk, Hk, 2), (nk, Hk, 3)))
    qo, ko = offsets(nq), offsets(nk)
    ref = prompt_reference(q, k, v, qo, ko, True, D ** -0.5)
    hurt = v.clone()
    n = nk[0]
    for at, col, value in ((n - 1, 7, "inf"), (n - 1, 8, "nan"), (n - 2, 7, "-inf"), (n - 5, 0, "nan"), (n - 9, 31, "inf"),
                           (n // 2, D - 1, "-inf"), (n // 2 + 3, D - 2, "inf"), (3, 5, "inf"), (n - 3, 5, "nan")):
        hurt[at, 1, col] = float(value)
    a = moe.Attention(H, Hk, D, BF16)
    out = a.prompt(q, k, hurt, i32(qo, DEV), i32(ko, DEV))
    assert a.device_status() == (moe.MOE_OK, 0)
    check(out[:, :2], None, tuple(x[:, :2] for x in ref), max(nk), D, BF16)  # the other key/value head
    check(out[nq[0]:], None, tuple(x[nq[0]:] for x in ref), max(nk), D, BF16)  # the other sequences
    got, bad = f64(out[:, 2:]), f64(hurt[:, 1])
    for t in range(nq[0]):
        seen = bad[:t + 1 + nk[0] - nq[0]]
        odd = ~np.isfinite(seen).all(0)
        for h in range(2):
            # (a weight of 0 times an infinity is NaN where all the row's keys were multiplied at once)
            assert not np.isfinite(got[t, h, odd]).any()
            assert np.isfinite(got[t, h, ~odd]).all(), (t, h)
    fine = np.isfinite(got)
    keep = np.where(fine, got, ref[0][:, 2:])  # the finite ones are right
    check(torch.from_numpy(keep), None, tuple(x[:, 2:] for x in ref), max(nk), D, BF16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("where", ["first", "late", "column", "all"])
def test_prompt_with_non_finite_values_takes_no_waits_to_their_limit(where, D, monkeypatch):
    """Rows that are not finite are not all computed again: a call with waits of at most 20 ms ends without an error."""
    monkeypatch.setenv("MOE_WAIT_TIMEOUT_MS", "20")
    T, H, Hk = 6000, 8, 2
    x = tensor((T, H + 2 * Hk, D), 1, BF16, DEV)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    at = {"first": (0, 5), "late": (T - 70, 5), "column": (slice(None), 5), "all": (slice(None), slice(None))}[where]
    v[at[0], 1, at[1]] = float("inf")
    a = moe.Attention(H, Hk, D, BF16)
    out = a.prompt(q, k, v, i32([0, T], DEV))
    assert a.device_status() == (moe.MOE_OK, 0)
    assert torch.isfinite(out[:, :4]).all()
    first = {"late": T - 70}.get(where, 0)
    assert not torch.isfinite(out[first:, 4:, 5]).any() and torch.isfinite(out[:first, 4:]).all()
    if where != "all":
        out[:, 4:, 5] = 0
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------------------------------------------------- scales

@pytest.mark.parametrize("scale", [1e-30, 1e-38, 3e-39, 1e-44])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 200), (F32, 64)])
def test_scales_near_zero(scale, dtype, D):
    """All weights are the same: a mean, and the logarithm of the number of keys."""
    scale = float(np.float32(scale))
    lens = [200, 70, 65, 64, 300, 64, 128]
    c, rows = make_cache(lens, 64, 16, 2, D, dtype)
    q = tensor((7, 4, D), 3, dtype, DEV)
    a = moe.Attention(4, 2, D, dtype, scale=scale)
    for shared in (0, 64):
        lse = torch.empty((7, 4), device=DEV)
        out = a.decode(q, c, i32(range(7), DEV), shared_len=shared, lse=lse)
        check(out, lse, decode_reference(q, c, rows, lens, 0, scale), 300, D, dtype)
    for nq, nk in (([150, 3], [150, 3]), ([7], [2500])):
        q, k, v = (tensor((sum(x), h, D), s, dtype, DEV) for x, h, s in ((nq, 4, 1), (nk, 2, 2), (nk, 2, 3)))
        lse = torch.empty((sum(nq), 4), device=DEV)
        out = a.prompt(q, k, v, i32(offsets(nq), DEV), i32(offsets(nk), DEV), lse=lse)
        check(out, lse, prompt_reference(q, k, v, offsets(nq), offsets(nk), True, scale), max(nk), D, dtype)
    assert a.device_status() == (moe.MOE_OK, 0)


# --------------------------------------------------------------------------------------------- the same, every time

@pytest.mark.parametrize("H,Hk,D", [(8, 2, 64), (16, 2, 128)])
def test_decode_repeats_itself_beside_other_work(H, Hk, D):
    """Bit for bit, whichever CTAs find an SM first: sums do not depend on who takes what."""
    lens = [32 + 5 + 23 * i for i in range(64)]
    c, _ = make_cache(lens, 32, 16, Hk, D, BF16)
    q, slots = tensor((64, H, D), 1, BF16, DEV), i32(range(64), DEV)
    a, b = moe.Attention(H, Hk, D, BF16), moe.Attention(8, 8, 64, BF16)
    want = a.decode(q, c, slots, shared_len=32)
    x = [tensor((t, 24, 64), 2, BF16, DEV) for t in (130, 700, 1500, 2900)]
    o = [i32([0, t], DEV) for t in (130, 700, 1500, 2900)]
    outs = [torch.empty_like(want) for _ in range(400)]
    other, y = torch.cuda.Stream(), [torch.empty((len(z), 8, 64), dtype=BF16, device=DEV) for z in x]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        j = i % 4
        b.prompt(x[j][:, :8], x[j][:, 8:16], x[j][:, 16:], o[j], out=y[j], stream=other)
        a.decode(q, c, slots, shared_len=32, out=out)
    torch.cuda.synchronize()
    assert sum(not torch.equal(out, want) for out in outs) == 0


# ---------------------------------------------------------------------------------------------------- wide tables

@pytest.mark.parametrize("shared", [0, 256])
def test_decode_with_tables_for_very_long_sequences(shared):
    """A table that could hold 2^30 positions a slot: slices are smaller, so that their counts stay below 2^32."""
    n, page = 100, 256
    lens = [shared + 3 * i for i in range(n)]
    lens[64] = 0
    c, rows = make_cache(lens, shared, page, 1, 8, BF16)
    table = torch.full((n, 1 << 22), -1, dtype=torch.int32, device=DEV)
    table[:, :c.width] = c.table
    wide = moe.KVCache(c.k, c.v, table, c.lens, c.refs)
    trim(wide, lens)
    out, lse, q, st = decode(wide, 2, 8, BF16, range(n), shared)
    assert st == (moe.MOE_OK, 0)
    right(out, lse, q, c, rows, lens, list(range(n)), 8, BF16)


# ------------------------------------------------------------------------------ every key, one by one, in long sequences

def spikes(n, D, at, dtype):
    """n keys of which key j alone has a large product with query i where at[i] = j; values that tell keys apart."""
    g = torch.Generator().manual_seed(n)
    k = torch.randn((n, 1, D), generator=g)
    k = (8 * k / k.norm(dim=-1, keepdim=True)).to(dtype)
    v = torch.randn((n, 1, D), generator=g).to(dtype)
    return k, v, (4 * k[at, 0].float()).to(dtype)


# q . k is 256 for a query's own key and at most 256 cos of their angle for the others; with scale 1 the own key's weight is
# then 1 - n e^-(256 (1 - cos)). Among these directions the cosine stays below 0.61, so the others weigh less than 1e-40
# together: the result is the own key's value, exactly, and lse the own score, up to the D + 8 roundings of a sum of 256.

@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("n,causal", [(3000, False), (3000, True), (700, False)])
def test_prompt_finds_every_key(n, causal, D):
    """Each query's result is one key's value, and every key is the one of some query: none is lost or taken twice."""
    at = torch.arange(n) if causal else torch.randperm(n, generator=torch.Generator().manual_seed(1))
    for dtype in (BF16, F32):
        k, v, q = (x.to(DEV) for x in spikes(n, D, at, dtype))
        a = moe.Attention(1, 1, D, dtype, scale=1.0)
        lse = torch.empty((n, 1), device=DEV)
        out = a.prompt(q.unsqueeze(1), k, v, i32([0, n], DEV), causal=causal, lse=lse)
        assert torch.equal(out[:, 0], v[at.to(DEV), 0])
        want = (q.double() * k[at.to(DEV), 0].double()).sum(-1)
        assert ((lse[:, 0].double() - want).abs() <= (D + 8) * 2.0 ** -24 * want + 2.0 ** -20).all()
        few = a.prompt(q[-40:].unsqueeze(1), k, v, i32([0, 40], DEV), i32([0, n], DEV), causal=causal)  # split keys
        assert torch.equal(few[:, 0], v[at[-40:].to(DEV), 0])


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (200, BF16), (64, F32), (200, F32)])
@pytest.mark.parametrize("page,shared", [(16, 0), (64, 0), (16, 1264), (128, 1152)])
def test_decode_finds_every_key(page, shared, D, dtype):
    """Key after key of sequences of 1500 positions, through the pages, shared and own."""
    n, seqs = 1500, 60
    at = torch.arange(n)
    k, v, q = (x.to(DEV) for x in spikes(n, D, at, dtype))
    c, rows = make_cache([n] * seqs, shared, page, 1, D, dtype)
    for i, r in enumerate(rows):
        where = i32(r, DEV).long()
        for pool, x in ((c.k, k), (c.v, v)):
            full = torch.zeros((len(r) * page, D), dtype=dtype, device=DEV)
            full[:n] = x[:, 0]
            pool[0, where, 0] = full.view(len(r), page, D)
    a, slots = moe.Attention(1, 1, D, dtype, scale=1.0), i32(range(seqs), DEV)
    lse = torch.empty((seqs, 1), device=DEV)
    for first in range(0, n, seqs):
        out = a.decode(q[first:first + seqs].unsqueeze(1), c, slots, shared_len=shared, lse=lse)
        assert torch.equal(out[:, 0], v[first:first + seqs, 0]), first
        want = (q[first:first + seqs].double() * k[first:first + seqs, 0].double()).sum(-1)
        assert ((lse[:, 0].double() - want).abs() <= (D + 8) * 2.0 ** -24 * want + 2.0 ** -20).all()
    assert a.device_status() == (moe.MOE_OK, 0)


# ------------------------------------------------------------------------------------------- scores that are all -inf

@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 200), (F32, 64)])
def test_rows_whose_scores_are_all_minus_infinity_are_rows_that_see_nothing(dtype, D):
    T, H, Hk = 1500, 4, 2
    q = tensor((T, H, D), 1, dtype, DEV)
    q[..., 3] = 1.0
    k, v = tensor((T, Hk, D), 2, dtype, DEV), tensor((T, Hk, D), 3, dtype, DEV)
    k[:70, 1, 3] = float("-inf")  # (all that the first 70 rows see of this key/value head)
    a = moe.Attention(H, Hk, D, dtype)
    for tq in (T, 16):  # (16 rows: split keys)
        lo = T - tq
        qo, ko = i32([0, tq], DEV), i32([0, T], DEV)
        kk = k if tq == T else torch.cat([k[:70]] * (T // 70 + 1))[:T]
        lse = torch.zeros((tq, H), device=DEV)
        out = a.prompt(q[lo:].contiguous(), kk, v, qo, ko, lse=lse)
        none = 70 if tq == T else tq
        assert (out[:none, 2:] == 0).all() and torch.isneginf(lse[:none, 2:]).all()
        assert torch.isfinite(out).all() and torch.isfinite(lse[:, :2]).all() and torch.isfinite(lse[none:]).all()
    c, rows = make_cache([64, 70, 150], 64, 16, Hk, D, dtype)
    for p in rows[0][:4]:
        c.k[0, p, 1, :, 3] = float("-inf")
    for shared in (0, 64):
        lse = torch.zeros((3, H), device=DEV)
        out = a.decode(q[:3], c, i32(range(3), DEV), shared_len=shared, lse=lse)
        assert (out[0, 2:] == 0).all() and torch.isneginf(lse[0, 2:]).all()
        assert torch.isfinite(out).all() and torch.isfinite(lse[1:]).all() and torch.isfinite(lse[:, :2]).all()
    assert a.device_status() == (moe.MOE_OK, 0)
