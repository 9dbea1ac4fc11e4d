"""Attention of chunks of new tokens over the paged cache against an fp64 implementation of the formula."""
import random

import numpy as np
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import attend64, check, f64, i32, offsets, prompt_reference, random_lens, tensor

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def pool(lens, page, Hk, D, dtype, seed, layers=1, garbage=float("nan"), width=None):
    """A cache whose slots hold `lens` positions in shuffled pages; everything else in the pool is `garbage`. Returns it with
    the slots' keys and values [n, Hk, D]."""
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    order = list(range(sum(need) + 3))
    r.shuffle(order)
    width = width or max(1, max(need)) + 1
    k = torch.full((layers, len(order), Hk, page, D), garbage, dtype=dtype)
    v = k.clone()
    table, refs, at, held = [], [0] * len(order), 0, []
    for s, n in enumerate(lens):
        rows = order[at:at + need[s]]
        at += need[s]
        table.append(rows + [-1] * (width - need[s]))
        kk, vv = tensor((n, Hk, D), seed + 2 * s, dtype, "cpu"), tensor((n, Hk, D), seed + 2 * s + 1, dtype, "cpu")
        held.append((kk, vv))
        for j, p in enumerate(rows):
            refs[p] = 1
            part = min(page, n - j * page)
            k[layers - 1, p, :, :part] = kk[j * page:j * page + part].transpose(0, 1)
            v[layers - 1, p, :, :part] = vv[j * page:j * page + part].transpose(0, 1)
    cache = moe.KVCache(k.to(DEV), v.to(DEV), i32(table, DEV), i32(lens, DEV), i32(refs, DEV))
    return cache, held


def reference(q, held, slots, offs, causal, scale):
    """prompt_reference over the slots' keys laid side by side."""
    ks = torch.cat([held[s][0] for s in slots]) if slots else torch.zeros((0,) + held[0][0].shape[1:])
    vs = torch.cat([held[s][1] for s in slots]) if slots else ks
    return prompt_reference(q, ks, vs, offs, offsets([len(held[s][0]) for s in slots]), causal, scale)


def run_chunk(nq, nk, H, Hk, D, dtype, page=64, causal=True, seed=0, qscale=1.0, layers=1, slots=None, extra=0, width=None):
    cache, held = pool(nk, page, Hk, D, dtype, seed, layers, width=width)
    slots = list(range(len(nk))) if slots is None else slots
    T, offs = sum(nq), offsets(nq)
    x = tensor((T + extra, H + 2 * Hk, D), seed + 77, dtype, DEV, qscale)
    q = x[:, :H]
    a = moe.Attention(H, Hk, D, dtype)
    out = torch.full((T + extra, H, D), float("nan"), dtype=dtype, device=DEV)
    lse = torch.full((T + extra, H), float("nan"), dtype=F32, device=DEV)
    a.chunk(q, cache, i32(slots, DEV), i32(offs, DEV), layer=layers - 1, causal=causal, out=out, lse=lse)
    assert a.device_status() == (moe.MOE_OK, 0)
    check(out[:T], lse[:T], reference(q[:T], held, slots, offs, causal, D ** -0.5), max(nk + [1]), D, dtype)
    if extra:
        assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
def test_lengths(n, dtype):
    """A whole prompt as one chunk, and its last tokens behind the others."""
    run_chunk([n], [n], 4, 2, 64, dtype, page=16, seed=n)
    run_chunk([min(n, 3)], [n], 4, 2, 64, dtype, page=32, seed=n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [8, 24, 64, 72, 80, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("page", [16, 256])
def test_head_dims(page, D, dtype):
    run_chunk([70, 3], [300, 3], 4, 2, D, dtype, page=page, seed=D)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (8, 1), (12, 4), (14, 2), (16, 16), (130, 1)])
def test_head_groups(H, Hk, dtype):
    run_chunk([5, 40], [200, 40], H, Hk, 32, dtype, seed=H)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_pages(page, causal, dtype):
    """Lengths that end at, before and behind a page's and a tile's end."""
    run_chunk([1, 4, 1, 30, 1], [page, page + 1, page - 1, 3 * page + 7, 129], 4, 2, 64, dtype, page=page, causal=causal, seed=page)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seed", range(5))
def test_mixed(seed, causal, D, dtype):
    """Ragged batches: empty chunks, empty slots, chunks longer than what their slot holds (rows that see nothing)."""
    r = random.Random(seed)
    n = r.randint(1, 12)
    nq = [r.choice([0, 1, 1, 2, 5, r.randint(1, 90)]) for _ in range(n)]
    nk = [max(0, a + r.choice([0, 0, 5, 130, 700, -1, -7, -200])) for a in nq]
    run_chunk(nq, nk, 6, 2, D, dtype, page=r.choice([16, 64, 128]), causal=causal, seed=seed, layers=2, extra=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("nq,nk", [([3, 18, 0, 1], [1100, 700, 50, 2049]), ([16], [4096]), ([1, 1], [1, 300]), ([1], [3001]),
                                   ([70, 5], [600, 0]), ([64], [1025])])
def test_few_rows_many_keys(nq, nk, D, dtype):
    """Rows whose keys are split over CTAs."""
    run_chunk(nq, nk, 6, 2, D, dtype, page=16, seed=D)
    run_chunk(nq, nk, 6, 2, D, dtype, page=64, causal=False, seed=D, width=5000)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_sequences(dtype):
    r = random.Random(5)
    nq = [r.choice([0, 1, 1, 3]) for _ in range(500)]
    run_chunk(nq, [a + r.choice([0, 1, 40]) for a in nq], 4, 1, 64, dtype, page=16, seed=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [(77, 128), (50, 128, 128), (200, 128, 256, 1), (129, 127, 128)])
def test_short_sequences_behind_cut_blocks(lens, D):
    """Many items of one or two blocks for each CTA, whole blocks behind ones that the sequence's end cuts."""
    nk = [lens[i % len(lens)] for i in range(700)]
    run_chunk([1] * 700, nk, 8, 4, D, BF16, page=64, seed=2)


@pytest.mark.parametrize("nq,nk", [([1] * 30 + [200, 150] + [3] * 6, 2300), ([140] * 12 + [2] * 20, 1700),
                                   ([130] * 10 + [1] * 20 + [257, 129, 128], 500)])
def test_long_runs_of_both_kinds(nq, nk):
    """Items of one tile and of two, enough of them that a CTA has a run of either kind, and (the last) just not."""
    r = random.Random(nk)
    lens = [n + r.randint(nk - 200, nk) for n in nq]
    run_chunk(nq, lens, 32, 32, 16, BF16, page=64, seed=6)


@pytest.mark.parametrize("D", [16, 64, 72, 128])
@pytest.mark.parametrize("shift", [8, 16])
def test_outputs_and_scratch_at_any_16_bytes(shift, D):
    """Results whose rows, and pieces whose memory, begin at a multiple of 16 bytes and of no more."""
    H, Hk, nq, nk = 6, 2, [150, 1, 5, 40], [900, 1500, 300, 40]
    cache, held = pool(nk, 64, Hk, D, BF16, 3)
    T, offs = sum(nq), offsets(nq)
    q = tensor((T, H, D), 5, BF16, DEV)
    buf = torch.full((T * (H * D + shift) + shift,), float("nan"), dtype=BF16, device=DEV)
    out = buf[shift:].as_strided((T, H, D), (H * D + shift, D, 1))
    a = moe.Attention(H, Hk, D, BF16)
    s, o = i32([0, 1, 2, 3], DEV), i32(offs, DEV)
    a.chunk(q, cache, s, o, out=out)
    check(out, None, reference(q, held, [0, 1, 2, 3], offs, True, D ** -0.5), max(nk), D, BF16)
    assert torch.isnan(buf[:shift]).all()
    assert torch.isnan(buf[shift:].as_strided((T, shift), (H * D + shift, 1), H * D + shift)).all()
    need = a._lib.moe_attention_chunk_workspace_bytes(cache._ref, 4, T, H) - 256
    header = torch.zeros(256, dtype=torch.uint8, device=DEV)
    scratch = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)
    again = torch.zeros((T, H, D), dtype=BF16, device=DEV)
    for at in (16, 32, 48, 240):
        rc = a._lib.moe_attention_chunk_ex(cache._ref, 0, q.data_ptr(), s.data_ptr(), o.data_ptr(), 4, T, H, H * D, H * D,
                                           a.scale, 1, again.data_ptr(), None, header.data_ptr(), 256,
                                           scratch.data_ptr() + at, need, torch.cuda.current_stream().cuda_stream)
        assert rc == moe.MOE_OK
        assert torch.equal(again, out)
        again.zero_()
        torch.cuda.synchronize()
        assert (scratch[:at] == 0xff).all() and (scratch[at + need:] == 0xff).all()
    assert not header.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slots_in_any_order_and_twice(dtype):
    """Slots named in another order than the table's, some not at all, one by two sequences."""
    run_chunk([3, 20, 7, 1], [50, 300, 20, 131], 4, 2, 64, dtype, seed=4, slots=[3, 1, 0, 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [128, 256])
def test_large_scores(D, dtype):
    run_chunk([100, 2], [500, 700], 4, 2, D, dtype, seed=3, qscale=30.0)


def test_many_rows():
    """Several tile pairs a head, whose items the runs cut anywhere."""
    run_chunk([700, 1, 150], [900, 1500, 150], 8, 2, 128, BF16, seed=9)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nonfinite_stays_where_it_is_seen(dtype, value, D):
    """A value that is not finite at one position reaches the rows from there on, in its column, and no other."""
    nq, nk, page, H, Hk = [60, 3], [400, 90], 16, 4, 2
    for place in (380, 399, 345):
        cache, held = pool(nk, page, Hk, D, dtype, 1)
        col = D - 3
        cache.v[0, int(cache.table[0, place // page]), 1, place % page, col] = value
        q = tensor((63, H, D), 5, dtype, DEV)
        a = moe.Attention(H, Hk, D, dtype)
        out = a.chunk(q, cache, i32([0, 1], DEV), i32([0, 60, 63], DEV))
        first = place - 340
        bad = ~torch.isfinite(out)
        want = torch.zeros_like(bad)
        want[first:60, 2:, col] = True
        assert torch.equal(bad, want)
        ref = reference(q, held, [0, 1], [0, 60, 63], True, D ** -0.5)
        fixed = torch.where(bad, torch.tensor(ref[0], device=DEV).to(out.dtype), out)
        check(fixed, None, ref, 400, D, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_tables_are_recorded(dtype, D):
    """A slot or length out of range: its rows see nothing. A page out of range: recorded. Other sequences are right."""
    nq, nk, H, Hk, page = [4, 5, 6], [100, 200, 60], 4, 2, 16
    offs = offsets(nq)
    q = tensor((15, H, D), 5, dtype, DEV)
    for spoil in ("slot", "negative", "length", "page", "offsets"):
        cache, held = pool(nk, page, Hk, D, dtype, 1)
        slots, o = [0, 1, 2], list(offs)
        if spoil == "slot":
            slots[1] = 7
        elif spoil == "negative":
            slots[1] = -1
        elif spoil == "length":
            cache.lens[1] = 10 ** 9
        elif spoil == "page":
            cache.table[1, 3] = 10 ** 6
        else:
            o = [0, 4, 99, 15]
        a = moe.Attention(H, Hk, D, dtype)
        out = torch.full((15, H, D), 5.0, dtype=dtype, device=DEV)
        a.chunk(q, cache, i32(slots, DEV), i32(o, DEV), out=out)
        status, detail = a.device_status()
        assert status == moe.MOE_ERR_DEVICE_CHECK and (detail == 1 or spoil == "offsets" and detail in (1, 2))
        ref = reference(q, held, [0, 1, 2], offs, True, D ** -0.5)
        check(out[:4], None, tuple(x[:4] for x in ref), 200, D, dtype)
        if spoil == "offsets":
            assert (out[4:] == 5).all()
        else:
            check(out[9:], None, tuple(x[9:] for x in ref), 200, D, dtype)
        if spoil in ("slot", "negative", "length"):
            assert (out[4:9] == 0).all()


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_graph_and_repeats(dtype, D):
    """A recorded call replayed on other contents gives what a plain call gives, bit for bit, every time."""
    cache, held = pool([1000, 300, 40], 64, 2, D, dtype, 1)
    a = moe.Attention(4, 2, D, dtype)
    q, slots, offs = tensor((30, 4, D), 5, dtype, DEV), i32([0, 1, 2], DEV), i32([0, 1, 20, 30], DEV)
    out = torch.empty_like(q)
    a.chunk(q, cache, slots, offs, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.chunk(q, cache, slots, offs, out=out)
    for seed in (6, 7):
        q.copy_(tensor((30, 4, D), seed, dtype, DEV))
        offs.copy_(i32([0, 10, 11, 30], DEV))
        g.replay()
        torch.cuda.synchronize()
        first = out.clone()
        assert torch.equal(first, a.chunk(q, cache, slots, offs))
        assert torch.equal(first, a.chunk(q, cache, slots, offs))
    assert a.device_status() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pipeline(dtype):
    """A prompt in pieces, then drafted and single tokens, each appended (normed and turned) and attended, against the
    whole sequence's attention over keys turned at once."""
    H, Hk, D, page = 8, 2, 64, 16
    rope = moe.Rotary(D, scaling="turns", factor=4.0, original_len=128)
    a = moe.Attention(H, Hk, D, dtype)
    lens = [300, 77]
    cache = moe.KVCache.create(1, 40, page, 2, 512, Hk, D, dtype)
    x = [tensor((n, H + 2 * Hk, D), i, dtype, DEV) for i, n in enumerate(lens)]
    wq, wk = tensor((D,), 8, dtype, DEV), tensor((D,), 9, dtype, DEV)
    slots, at = i32([1, 0], DEV), [0, 0]  # sequence i is in slot 1 - i
    got = [[], []]
    for step in [(128, 0), (100, 70), (64, 1), (4, 2), (1, 1), (3, 3)]:
        pos = i32(at, DEV)
        cache.resize(slots, i32([p + n for p, n in zip(at, step)], DEV))
        y = torch.cat([x[i][at[i]:at[i] + step[i]] for i in range(2)])
        offs = i32(offsets(step), DEV)
        q = cache.append(y[:, H:H + Hk], y[:, H + Hk:], slots, offs, pos, rope, q=y[:, :H], q_weight=wq, k_weight=wk)
        o = a.chunk(q, cache, slots, offs)
        got[0].append(o[:step[0]])
        got[1].append(o[step[0]:])
        at = [p + n for p, n in zip(at, step)]
    assert at == lens and cache.device_status() == (moe.MOE_OK, 0) and a.device_status() == (moe.MOE_OK, 0)
    whole = torch.cat(x)
    pos = i32(list(range(300)) + list(range(77)), DEV)
    q, k = rope.apply(whole[:, :H], pos, whole[:, H:H + Hk], q_weight=wq, k_weight=wk)
    ref = prompt_reference(q, k, whole[:, H + Hk:], [0, 300, 377], [0, 300, 377], True, D ** -0.5)
    check(torch.cat(got[0] + got[1]), None, ref, 300, D, dtype)
