"""Attention over packed prompts and over the paged cache against an fp64 implementation of the formula."""
import random

import numpy as np
import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import (attend64, check, f64, i32, offsets, prompt_reference, random_lens, tensor)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def run_prompt(nq, nk, H, Hk, D, dtype, causal=True, seed=0, fused=False, qscale=1.0):
    Tq, Tk = sum(nq), sum(nk)
    if fused:
        x = tensor((Tq, H + 2 * Hk, D), seed, dtype, DEV)
        q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    else:
        q = tensor((Tq, H, D), seed, dtype, DEV, qscale)
        k, v = tensor((Tk, Hk, D), seed + 1, dtype, DEV), tensor((Tk, Hk, D), seed + 2, dtype, DEV)
    a = moe.Attention(H, Hk, D, dtype)
    qo, ko = offsets(nq), offsets(nk)
    out = torch.full((Tq, H, D), float("nan"), dtype=dtype, device=DEV)
    lse = torch.full((Tq, H), float("nan"), dtype=F32, device=DEV)
    a.prompt(q, k, v, i32(qo, DEV), None if fused else i32(ko, DEV), causal=causal, out=out, lse=lse)
    assert a.device_status() == (moe.MOE_OK, 0)
    check(out, lse, prompt_reference(q, k, v, qo, ko, causal, D ** -0.5), max(nk + [1]), D, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 127, 128, 129, 200, 256, 257, 385])
def test_prompt_lengths(n, dtype):
    run_prompt([n], [n], 4, 2, 64, dtype, seed=n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [8, 16, 24, 32, 56, 64, 72, 80, 96, 112, 128, 136, 192, 256])
def test_prompt_head_dims(D, dtype):
    run_prompt([70, 3], [70, 3], 4, 2, D, dtype, seed=D)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (3, 1), (8, 1), (12, 4), (14, 2), (16, 16), (40, 8), (130, 1), (300, 1)])
def test_prompt_head_groups(H, Hk, dtype):
    run_prompt([5, 40], [5, 40], H, Hk, 32, dtype, seed=H)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seed", range(6))
def test_prompt_packed_with_past(seed, causal, dtype):
    """Ragged sequences, zeros among them, more keys than queries or fewer (rows that see nothing)."""
    r = random.Random(seed)
    n = r.randint(1, 9)
    nq = random_lens(r, n, 150)
    nk = [max(0, a + r.choice([0, 0, 5, 130, 300, -1, -7, -200])) for a in nq]
    run_prompt(nq, nk, 6, 2, r.choice([64, 128]), dtype, causal, seed)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("nq,nk", [([3, 18, 0, 1], [1100, 700, 50, 2049]), ([16], [4096]), ([1, 1], [1, 300]),
                                   ([70, 5], [600, 0]), ([64], [1025])])
def test_prompt_few_rows_many_keys(nq, nk, D, dtype):
    """Few tiles of rows: their keys are split over CTAs, some of which see none."""
    run_prompt(nq, nk, 6, 2, D, dtype, seed=D)
    run_prompt(nq, nk, 6, 2, D, dtype, causal=False, seed=D)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_no_keys_at_all(dtype):
    q = tensor((7, 4, 64), 1, dtype, DEV)
    kv = torch.empty((0, 2, 64), dtype=dtype, device=DEV)
    a = moe.Attention(4, 2, 64, dtype)
    lse = torch.zeros((7, 4), device=DEV)
    out = a.prompt(q, kv, kv, i32([0, 3, 7], DEV), i32([0, 0, 0], DEV), lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_strided_inputs(dtype):
    run_prompt([33, 100, 1], [33, 100, 1], 8, 2, 64, dtype, fused=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_many_short_sequences(dtype):
    r = random.Random(5)
    run_prompt(*(2 * [random_lens(r, 300, 4, 0.3)]), 4, 1, 64, dtype, seed=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_large_scores(dtype):
    """Scores in the hundreds: each row's softmax is nearly one key, and the running maximum moves often."""
    run_prompt([300], [300], 4, 2, 128, dtype, seed=3, qscale=30.0)


def test_prompt_rising_scores():
    """Scores that grow along the keys by far more than a rescaling threshold in every block."""
    n, D = 700, 64
    q = torch.zeros((n, 2, D), dtype=BF16, device=DEV)
    q[:, :, 0] = 8.0
    k = torch.zeros((n, 1, D), dtype=BF16, device=DEV)
    k[:, 0, 0] = torch.arange(n, device=DEV).to(BF16) * 0.5
    v = tensor((n, 1, D), 4, BF16, DEV)
    a = moe.Attention(2, 1, D, BF16, scale=1.0)
    lse = torch.empty((n, 2), device=DEV)
    out = a.prompt(q, k, v, i32([0, n], DEV), lse=lse)
    check(out, lse, prompt_reference(q, k, v, [0, n], [0, n], True, 1.0), n, D, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_nonfinite_stays_where_it_is_seen(value, D, dtype):
    """A non-finite key or value reaches no row that does not see its position: not the rows before it, not the
    neighbouring sequences."""
    lens, H, Hk = [50, 150, 60], 4, 2
    T, at = sum(lens), 50 + 90
    q, k, v = tensor((T, H, D), 1, dtype, DEV), tensor((T, Hk, D), 2, dtype, DEV), tensor((T, Hk, D), 3, dtype, DEV)
    o = offsets(lens)
    ref = prompt_reference(q, k, v, o, o, True, D ** -0.5)
    a = moe.Attention(H, Hk, D, dtype)
    keep = [t for t in range(T) if not at <= t < 200]
    for bad in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        (kk if bad == "k" else vv)[at, 1, 5] = value
        out = a.prompt(q, kk, vv, i32(o, DEV))
        sub = tuple(x[keep] for x in ref)
        check(out[keep], None, sub, 150, D, dtype)
        # the other key/value head's rows see nothing of it
        check(out[:, :2], None, tuple(x[:, :2] for x in ref), 150, D, dtype)
        if bad == "v":
            assert not torch.isfinite(out[at:200, 2:, 5]).any()
            hurt = out[at:200, 2:].clone()
            hurt[..., 5] = 0
            assert torch.isfinite(hurt).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
def test_prompt_split_keys_nonfinite(value, dtype):
    """The same where the keys of few rows are split over CTAs: a position that some rows do not see, in the last part."""
    nq, nk, H, Hk, D = [8, 20, 1], [2000, 900, 1200], 4, 2, 128
    Tq, Tk, at = sum(nq), sum(nk), 2000 - 3  # seen by the last three tokens of sequence 0
    q = tensor((Tq, H, D), 1, dtype, DEV)
    k, v = tensor((Tk, Hk, D), 2, dtype, DEV), tensor((Tk, Hk, D), 3, dtype, DEV)
    qo, ko = offsets(nq), offsets(nk)
    ref = prompt_reference(q, k, v, qo, ko, True, D ** -0.5)
    a = moe.Attention(H, Hk, D, dtype)
    keep = [t for t in range(Tq) if not 5 <= t < 8]
    for bad in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        (kk if bad == "k" else vv)[at, 1, 5] = value
        out = a.prompt(q, kk, vv, i32(qo, DEV), i32(ko, DEV))
        check(out[keep], None, tuple(x[keep] for x in ref), 2000, D, dtype)
        check(out[:, :2], None, tuple(x[:, :2] for x in ref), 2000, D, dtype)
        if bad == "v":
            assert not torch.isfinite(out[5:8, 2:, 5]).any()
            hurt = out[5:8, 2:].clone()
            hurt[..., 5] = 0
            assert torch.isfinite(hurt).all()
    assert a.device_status()[0] == moe.MOE_OK


def test_prompt_split_keys_bad_offsets():
    """A sequence with bad offsets is recorded and its rows stay as they were; the others are computed."""
    q, kv = tensor((24, 4, 64), 1, BF16, DEV), tensor((3000, 2, 64), 2, BF16, DEV)
    a = moe.Attention(4, 2, 64, BF16)
    for qo, ko, bad, rows in [([0, 8, 24], [0, 3001, 3000], (0, 1), range(0, 24)), ([0, 8, 25], [0, 1500, 3000], (1,), range(8, 24)),
                              ([0, 8, 24], [0, 1500, 3004], (1,), range(8, 24))]:
        out = torch.full((24, 4, 64), 7.0, dtype=BF16, device=DEV)
        a.prompt(q, kv, kv, i32(qo, DEV), i32(ko, DEV), out=out)
        st, seq = a.device_status()
        assert st == moe.MOE_ERR_DEVICE_CHECK and seq in bad  # (of two, whichever is found first)
        assert (out[list(rows)] == 7).all()
        good = [t for t in range(24) if t not in rows]
        if good:
            ref = prompt_reference(q[good], kv[:1500], kv[:1500], [0, 8], [0, 1500], True, 64 ** -0.5)
            check(out[good], None, ref, 1500, 64, BF16)


def test_prompt_split_keys_with_little_workspace_and_in_a_graph():
    nq, nk, H, Hk, D = [3, 40], [2500, 1000], 8, 2, 64
    q, kv = tensor((43, H, D), 1, BF16, DEV), tensor((3500, Hk, D), 2, BF16, DEV)
    qo, ko = offsets(nq), offsets(nk)
    ref = prompt_reference(q, kv, kv, qo, ko, True, D ** -0.5)
    a = moe.Attention(H, Hk, D, BF16)
    lse = torch.empty((43, H), device=DEV)
    first = a.prompt(q, kv, kv, i32(qo, DEV), i32(ko, DEV), lse=lse)
    check(first, lse, ref, 2500, D, BF16)
    need = a._lib.moe_attention_prompt_workspace_bytes(2, 43, 3500, H, Hk, D, moe.MOE_DTYPE_BF16)
    assert need > 256
    # a workspace of the least size: the same numbers without the split
    ws, out = torch.zeros(need - 1, dtype=torch.uint8, device=DEV), torch.empty_like(first)
    stream = torch.cuda.current_stream().cuda_stream
    oq, ok = i32(qo, DEV), i32(ko, DEV)
    for nbytes in (256, need - 1):
        out.fill_(0)
        assert a._lib.moe_attention_prompt(q.data_ptr(), kv.data_ptr(), kv.data_ptr(), oq.data_ptr(), ok.data_ptr(), 2, 43, 3500,
                                           H, Hk, D, H * D, Hk * D, Hk * D, H * D, D ** -0.5, 1, moe.MOE_DTYPE_BF16,
                                           out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nbytes, stream) == moe.MOE_OK
        check(out, lse, ref, 2500, D, BF16)
    g, o = torch.cuda.CUDAGraph(), torch.zeros_like(first)
    with torch.cuda.graph(g):
        a.prompt(q, kv, kv, oq, ok, out=o)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)
    assert a.device_status()[0] == moe.MOE_OK


def test_prompt_bad_offsets_are_recorded():
    q, kv = tensor((20, 4, 64), 1, BF16, DEV), tensor((20, 2, 64), 2, BF16, DEV)
    a = moe.Attention(4, 2, 64, BF16)
    for qo, ko, seq in [([0, 8, 21], None, 1), ([0, 12, 8], None, 1), ([0, 8, 20], [0, 25, 20], 0), ([-4, 8, 20], None, 0)]:
        a.prompt(q, kv, kv, i32(qo, DEV), None if ko is None else i32(ko, DEV))
        st, _ = a.device_status()
        assert st == moe.MOE_ERR_DEVICE_CHECK
    out = a.prompt(q, kv, kv, i32([0, 20], DEV))
    assert a.device_status() == (moe.MOE_OK, 0)
    check(out, None, prompt_reference(q, kv, kv, [0, 20], [0, 20], True, 0.125), 20, 64, BF16)


# ------------------------------------------------------------------------------------------------ decode

def make_cache(lens, shared, page, Hk, D, dtype, layers=1, seed=0, stale=0.0):
    """A cache whose slots share their first `shared` positions, on shuffled pages; stale: what unused positions hold."""
    r = random.Random(seed)
    up = lambda a: -(-a // page)  # noqa: E731
    pages = up(shared) + sum(max(0, up(a) - shared // page) for a in lens) + 3
    order = list(range(pages))
    r.shuffle(order)
    head, at = order[:shared // page], shared // page
    rows = []
    for a in lens:
        need = max(0, up(a) - shared // page)
        rows.append(head + order[at:at + need])
        at += need
    width = max(len(x) for x in rows) + 1
    k = tensor((layers, pages, Hk, page, D), seed + 1, dtype, "cpu")
    v = tensor((layers, pages, Hk, page, D), seed + 2, dtype, "cpu")
    used = torch.zeros((pages, page), dtype=torch.bool)
    for x, a in zip(rows, lens):
        for p in range(a):
            used[x[p // page], p % page] = True
    hide = ~used[None, :, None, :, None]
    if stale:
        k, v = k.masked_fill(hide, stale), v.masked_fill(hide, stale)
    refs = [0] * pages
    for x in rows:
        for p in x:
            refs[p] += 1
    c = moe.KVCache(k.to(DEV), v.to(DEV), i32([x + [-1] * (width - len(x)) for x in rows], DEV), i32(lens, DEV),
                    i32(refs, DEV))
    return c, rows


def decode_reference(q, c, rows, lens, layer, scale):
    n, H, D = q.shape
    k, v = c.k[layer].cpu(), c.v[layer].cpu()
    got = []
    for i in range(n):
        at = torch.tensor(rows[i], dtype=torch.long)
        kk, vv = (f64(x[at].transpose(1, 2).reshape(-1, x.shape[1], D)[:lens[i]]) for x in (k, v))
        got.append(attend64(f64(q[i:i + 1]), kk, vv, [lens[i]], scale))
    return tuple(np.concatenate([g[j] for g in got]) for j in range(4))


def run_decode(lens, shared, H, Hk, D, dtype, page=16, layers=1, layer=0, seed=0, stale=0.0, use=None):
    c, rows = make_cache(lens, shared, page, Hk, D, dtype, layers, seed, stale)
    n = len(lens)
    q = tensor((n, H + 3, D), seed + 9, dtype, DEV)[:, :H]
    a = moe.Attention(H, Hk, D, dtype)
    out = torch.full((n, H, D), float("nan"), dtype=dtype, device=DEV)
    lse = torch.full((n, H), float("nan"), device=DEV)
    a.decode(q, c, i32(list(range(n)), DEV), layer=layer, shared_len=shared if use is None else use, out=out, lse=lse)
    assert a.device_status() == (moe.MOE_OK, 0)
    check(out, lse, decode_reference(q, c, rows, lens, layer, D ** -0.5), max(lens + [1]), D, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 2000])
def test_decode_lengths(n, dtype):
    run_decode([n], 0, 8, 2, 64, dtype, seed=n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [8, 24, 64, 80, 96, 128, 136, 256])
def test_decode_head_dims(D, dtype):
    run_decode([70, 3, 40], 32, 4, 2, D, dtype, seed=D)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (7, 1), (8, 1), (16, 2), (17, 1), (40, 2), (64, 8), (130, 1)])
def test_decode_head_groups(H, Hk, dtype):
    run_decode([150, 40, 97], 32, H, Hk, 64, dtype, seed=H)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(page, dtype):
    run_decode([4 * page + 5, 3 * page, 3 * page + 1, 6 * page - 1], 3 * page, 8, 2, 64, dtype, page, layers=2, layer=1,
               seed=page)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("seed", range(8))
def test_decode_ragged(seed, dtype):
    r = random.Random(seed)
    shared = 16 * r.choice([0, 1, 7, 8, 9, 40])
    lens = [shared + r.choice([0, 1, 16, r.randint(0, 700)]) for _ in range(r.choice([1, 2, 9, 33, 70]))]
    run_decode(lens, shared, *r.choice([(8, 2), (8, 8), (12, 2)]), r.choice([64, 128]), dtype, seed=seed)


@pytest.mark.parametrize("H,Hk,D,page", [(8, 8, 64, 16), (16, 8, 128, 64), (64, 4, 128, 32), (128, 8, 64, 128)])
def test_decode_long_runs(H, Hk, D, page):
    """Enough keys that every CTA walks many blocks of several sequences, its ring round and round."""
    r = random.Random(H)
    shared = 2 * page
    lens = [shared + r.choice([0, 1, 63, 64, 65, r.randint(500, 1900), r.randint(1000, 1900)]) for _ in range(40)]
    run_decode(lens, shared, H, Hk, D, BF16, page, seed=H)


def test_decode_many_rows_of_one_head():
    """More rows of a key/value head than one tile of the shared part holds."""
    run_decode([160 + i % 7 for i in range(80)], 144, 16, 2, 64, BF16)


def test_decode_shares_less_than_it_could():
    """shared_len may say less than what the slots really share, or nothing."""
    for use in (0, 16, 64):
        run_decode([100, 150, 97], 96, 8, 2, 128, BF16, use=use)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stale", [float("nan"), float("inf")])
def test_decode_unused_positions_do_not_matter(stale, dtype):
    run_decode([33, 70, 48, 100, 0], 0, 8, 2, 64, dtype, stale=stale)
    run_decode([33, 70, 48, 100, 32], 32, 8, 2, 128, dtype, stale=stale)


def test_decode_long_cache_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: offsets of its last pages need 64 bits."""
    page, Hk, D = 256, 8, 128
    pages = (1 << 31) // (page * Hk * D) + 40
    c = moe.KVCache.create(1, pages, page, 2, 8 * page, Hk, D, BF16, DEV)
    for x, s in ((c.k, 1), (c.v, 2)):
        x[:, -40:] = tensor((1, 40, Hk, page, D), s, BF16, DEV)
    rows = [list(range(pages - 1, pages - 9, -1)), list(range(pages - 1, pages - 5, -1)) + list(range(pages - 20, pages - 16))]
    c.table.copy_(i32(rows, DEV))
    lens = [8 * page - 3, 7 * page + 9]
    c.lens.copy_(i32(lens, DEV))
    q = tensor((2, 16, D), 3, BF16, DEV)
    a = moe.Attention(16, Hk, D, BF16)
    for shared in (0, 4 * page):
        out = a.decode(q, c, i32([0, 1], DEV), shared_len=shared)
        k, v = c.k[0, -40:].cpu(), c.v[0, -40:].cpu()
        for i in range(2):
            at = torch.tensor(rows[i]) - (pages - 40)
            kk, vv = (f64(x[at].transpose(1, 2).reshape(-1, Hk, D)[:lens[i]]) for x in (k, v))
            check(out[i:i + 1], None, attend64(f64(q[i:i + 1]), kk, vv, [lens[i]], D ** -0.5), lens[i], D, BF16)


def test_decode_bad_tables_are_recorded():
    c, rows = make_cache([60, 60, 60], 32, 16, 2, 64, BF16)
    q = tensor((3, 8, 64), 5, BF16, DEV)
    a = moe.Attention(8, 2, 64, BF16)
    ref = decode_reference(q, c, rows, [60] * 3, 0, 0.125)
    # a slot out of range: its rows are 0, the others are right
    out = a.decode(q, c, i32([0, 7, 2], DEV), shared_len=32)
    assert a.device_status() == (moe.MOE_ERR_DEVICE_CHECK, 1)
    assert (out[1] == 0).all()
    check(out[[0, 2]], None, tuple(x[[0, 2]] for x in ref), 60, 64, BF16)
    # a page out of range
    c.table[2, 3] = 1 << 20
    a.decode(q, c, i32([0, 1, 2], DEV), shared_len=32)
    assert a.device_status() == (moe.MOE_ERR_DEVICE_CHECK, 2)


def test_prompt_is_deterministic_and_graph_replays():
    q, kv = tensor((500, 8, 128), 1, BF16, DEV), tensor((500, 2, 128), 2, BF16, DEV)
    o = i32([0, 200, 500], DEV)
    a = moe.Attention(8, 2, 128, BF16)
    first = a.prompt(q, kv, kv, o)
    out = torch.zeros_like(first)
    with moe.GraphCapture(keep=(q, kv, o, out, a)) as cap:
        a.prompt(q, kv, kv, o, out=out, stream=cap.stream)
    for _ in range(3):
        out.zero_()
        cap.graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_decode_is_deterministic_on_two_streams_and_in_a_graph():
    lens = [900 + 37 * i for i in range(8)]
    c, _ = make_cache(lens, 512, 32, 2, 128, BF16)
    q = tensor((8, 16, 128), 1, BF16, DEV)
    slots = i32(list(range(8)), DEV)
    a = moe.Attention(16, 2, 128, BF16)
    first = a.decode(q, c, slots, shared_len=512)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        o = torch.empty_like(first)
        outs.append(o)
        streams[i % 2].wait_stream(torch.cuda.current_stream())
        a.decode(q, c, slots, shared_len=512, out=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    g, o = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(g):
        a.decode(q, c, slots, shared_len=512, out=o)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)


def test_binding_refuses_on_the_gpu():
    q, kv = tensor((8, 4, 64), 1, BF16, DEV), tensor((8, 2, 64), 2, BF16, DEV)
    o = i32([0, 8], DEV)
    a = moe.Attention(4, 2, 64, BF16)
    for args in [(q[:, :3], kv, kv, o), (q, kv[:7], kv, o), (q, kv[:7], kv[:7], o), (q.float(), kv, kv, o),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), kv, kv, o), (q, kv, kv, o.long()), (q, kv, kv, o.cpu()),
                 (q, kv, kv, o[:0])]:
        with pytest.raises(ValueError):
            a.prompt(*args)
    with pytest.raises(ValueError):
        a.prompt(q, kv, kv, o, out=torch.empty((7, 4, 64), dtype=BF16, device=DEV))
    with pytest.raises(moe.MoeError):  # a stride that is no multiple of 16 bytes
        x = torch.zeros((8, 4 * 64 + 4), dtype=BF16, device=DEV)
        a.prompt(x[:, :256].unflatten(1, (4, 64)), kv, kv, o)


def test_workspace_needs_only_its_header_prepared():
    c, _ = make_cache([300, 1, 0, 77], 64, 32, 2, 64, BF16)
    q, slots = tensor((4, 8, 64), 1, BF16, DEV), i32([0, 1, 2, 3], DEV)
    kv, o = tensor((40, 2, 64), 2, BF16, DEV), i32([0, 40], DEV)
    qp = tensor((40, 8, 64), 3, BF16, DEV)
    a = moe.Attention(8, 2, 64, BF16)

    def all_calls():
        return [a.decode(q, c, slots), a.decode(q, c, slots, shared_len=64), a.prompt(qp, kv, kv, o)]

    first = all_calls()
    for t, _, _ in a._ws._of.values():
        t[256:].fill_(255)
    for x, y in zip(first, all_calls()):
        assert torch.equal(x, y)
    assert a.device_status()[0] == moe.MOE_OK


def test_recorded_calls_share_one_workspace_of_their_own():
    c, _ = make_cache([900, 33, 64], 32, 32, 2, 128, BF16)
    q, slots = tensor((3, 8, 128), 1, BF16, DEV), i32([0, 1, 2], DEV)
    a = moe.Attention(8, 2, 128, BF16)
    want = a.decode(q, c, slots)
    need = a._ws._of[torch.cuda.current_stream().cuda_stream][1]
    assert a._lib.moe_stream_capture_id(torch.cuda.current_stream().cuda_stream) == 0
    graphs = []
    for _ in range(2):
        outs = [torch.empty_like(want) for _ in range(6)]
        g, before = torch.cuda.CUDAGraph(), torch.cuda.memory_allocated()
        with torch.cuda.graph(g):
            for o in outs:
                a.decode(q, c, slots, out=o)
        assert torch.cuda.memory_allocated() - before < 2 * need  # one workspace (and what torch keeps for a graph)
        graphs.append((g, outs))
    assert a.device_status()[0] == moe.MOE_OK  # nothing has run yet
    spaces = {w[2] for w in a._ws._recorded.values()} | {w[2] for w in a._ws._of.values()}
    assert len(spaces) == 3
    # both graphs and eager calls at once, on three streams
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        assert torch.equal(a.decode(q, c, slots), want)
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(o, want) for o in outs)
    assert a.device_status()[0] == moe.MOE_OK
    slots[1] = 99  # no such slot: a recorded call reports it
    graphs[0][0].replay()
    assert a.device_status() == (moe.MOE_ERR_DEVICE_CHECK, 1)
    assert a.device_status()[0] == moe.MOE_OK


def test_recordings_one_after_the_other_on_private_streams():
    q, kv = tensor((70, 4, 64), 1, BF16, DEV), tensor((70, 2, 64), 2, BF16, DEV)
    o = i32([0, 70], DEV)
    a = moe.Attention(4, 2, 64, BF16)
    want, caps = a.prompt(q, kv, kv, o), []
    for _ in range(3):
        out = torch.zeros_like(want)
        with moe.GraphCapture(keep=(q, kv, o, out, a)) as cap:
            a.prompt(q, kv, kv, o, out=out, stream=cap.stream)
        caps.append((cap, out))
    assert len({w[2] for w in a._ws._recorded.values()}) == 3
    for cap, out in caps:
        cap.graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert a.device_status()[0] == moe.MOE_OK


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [136, 256])
@pytest.mark.parametrize("lens", [[50, 150, 60], [50, 150, 60] * 12, [700, 900]])
def test_prompt_long_heads_nonfinite(lens, D, value):
    """Heads of more than 128: a non-finite key or value reaches only rows that see it, with and without split keys."""
    H, Hk, n0, n1 = 4, 2, lens[0], lens[1]
    T, at = sum(lens), lens[0] + n1 - 60
    q, k, v = tensor((T, H, D), 1, BF16, DEV), tensor((T, Hk, D), 2, BF16, DEV), tensor((T, Hk, D), 3, BF16, DEV)
    o = offsets(lens)
    ref = prompt_reference(q, k, v, o, o, True, D ** -0.5)
    a = moe.Attention(H, Hk, D, BF16)
    keep = [t for t in range(T) if not at <= t < n0 + n1]
    for bad in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        (kk if bad == "k" else vv)[at, 1, 5] = value
        out = a.prompt(q, kk, vv, i32(o, DEV))
        check(out[keep], None, tuple(x[keep] for x in ref), max(lens), D, BF16)
        check(out[:, :2], None, tuple(x[:, :2] for x in ref), max(lens), D, BF16)
        if bad == "v":
            assert not torch.isfinite(out[at:n0 + n1, 2:, 5]).any()
            hurt = out[at:n0 + n1, 2:].clone()
            hurt[..., 5] = 0
            assert torch.isfinite(hurt).all()
    assert a.device_status()[0] == moe.MOE_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [136, 192, 200, 256])
def test_decode_long_heads_with_shared_tiles(D, dtype):
    """Enough sequences that the shared positions go to tiles: rows that fill one and rows that do not, short slots."""
    run_decode([100, 96, 31, 0, 97, 200], 96, 8, 2, D, dtype, seed=D)
    run_decode([300 + 3 * i for i in range(20)], 288, 8, 1, D, dtype, page=32, seed=D)
    run_decode([1100, 1040, 1025, 1300, 1024, 1030, 1100], 1024, 4, 4, D, dtype, page=64, layers=2, layer=1, seed=D)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [128, 192, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_decode_shared_nonfinite_and_short_slots(value, D, dtype):
    """A non-finite value at a shared position reaches no slot that ends before it."""
    lens, shared, H, Hk, page = [150, 90, 128, 140, 64, 128, 150], 128, 8, 2, 16
    c, rows = make_cache(lens, shared, page, Hk, D, dtype)
    n, at = len(lens), 100
    q = tensor((n, H, D), 9, dtype, DEV)
    ref = decode_reference(q, c, rows, lens, 0, D ** -0.5)
    c.v[0, rows[0][at // page], 1, at % page, 5] = value
    a = moe.Attention(H, Hk, D, dtype)
    out = a.decode(q, c, i32(list(range(n)), DEV), shared_len=shared)
    short = [1, 4]
    check(out[short], None, tuple(x[short] for x in ref), 150, D, dtype)
    check(out[:, :4], None, tuple(x[:, :4] for x in ref), 150, D, dtype)
    seen = out[[0, 2, 3, 5, 6], 4:].clone()
    assert not torch.isfinite(seen[..., 5]).any()
    seen[..., 5] = 0
    assert torch.isfinite(seen).all()
    assert a.device_status()[0] == moe.MOE_OK
