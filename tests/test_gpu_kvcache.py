"""The paged cache's calls against the same bookkeeping on plain lists: tables, counts and every page's bits."""
import random

import pytest
import torch

import sparse_mixture_experts_moe_gb300 as moe
from attention_cases import Model, attend64, check, f64, i32, offsets, tensor

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def pair(layers=2, pages=60, page=16, slots=10, width=12, Hk=2, D=32, dtype=BF16, seed=0):
    c = moe.KVCache.create(layers, pages, page, slots, width * page, Hk, D, dtype, DEV)
    c.k.copy_(tensor(c.k.shape, seed + 1, dtype, DEV))
    c.v.copy_(tensor(c.v.shape, seed + 2, dtype, DEV))
    m = Model(layers, pages, page, slots, width)
    m.k, m.v = c.k.cpu(), c.v.cpu()
    return c, m


def same(c, m):
    assert c.table.tolist() == m.table()
    assert c.lens.tolist() == m.lens
    assert c.refs.tolist() == m.refs
    assert torch.equal(c.k.cpu(), m.k) and torch.equal(c.v.cpu(), m.v)


def resize(c, m, slots, lens):
    c.resize(i32(slots, DEV), i32(lens, DEV))
    bad = m.resize(slots, lens)
    st, detail = c.device_status()
    assert (st == moe.MOE_ERR_DEVICE_CHECK and detail in bad) if bad else st == moe.MOE_OK
    same(c, m)


def fork(c, m, src, dst):
    c.fork(i32(src, DEV), i32(dst, DEV))
    bad = m.fork(src, dst)
    st, detail = c.device_status()
    assert (st == moe.MOE_ERR_DEVICE_CHECK and detail in bad) if bad else st == moe.MOE_OK
    same(c, m)


def compact(c, m):
    live = c.compact()
    assert live.tolist() == [m.compact()]
    assert c.device_status() == (moe.MOE_OK, 0)
    same(c, m)


def write(c, m, layer, slots, counts, pos, seed):
    k = tensor((sum(counts), c.kv_heads + 1, c.head_dim), seed, c.dtype, DEV)[:, :c.kv_heads]
    v = tensor((sum(counts), c.kv_heads, c.head_dim), seed + 1, c.dtype, DEV)
    o = offsets(counts)
    c.write(k, v, i32(slots, DEV), i32(o, DEV), i32(pos, DEV), layer=layer)
    assert c.device_status() == (moe.MOE_OK, 0)
    m.write(layer, slots, o, pos, k.cpu(), v.cpu())
    same(c, m)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_grow_write_shrink(page, dtype):
    c, m = pair(page=page, dtype=dtype, pages=30, width=6, D=40)
    resize(c, m, [3, 0, 7], [page, 1, 2 * page + 5])
    write(c, m, 1, [3, 0, 7], [page, 1, 2 * page + 5], [0, 0, 0], 5)
    resize(c, m, [0, 7], [page + 1, page])
    write(c, m, 0, [0], [page], [1], 6)
    resize(c, m, [7, 3, 0], [0, 6 * page, page + 1])
    resize(c, m, [1, 2], [1, 0])


def test_fork_shares_and_copies():
    c, m = pair()
    resize(c, m, [0, 1], [37, 32])
    write(c, m, 0, [0, 1], [37, 32], [0, 0], 3)
    write(c, m, 1, [0, 1], [37, 32], [0, 0], 4)
    fork(c, m, [0, 0, 1, 9], [2, 3, 4, 5])  # a partial page, twice; a full one; an empty slot
    resize(c, m, [2, 3, 4, 0], [38, 50, 33, 38])
    write(c, m, 0, [2, 3, 4, 0], [1, 13, 1, 1], [37, 37, 32, 37], 9)
    fork(c, m, [2, 4], [0, 3])  # over slots that hold something
    resize(c, m, [0, 1, 2, 3, 4], [0] * 5)
    assert m.refs == [0] * 60


def test_growing_after_truncation_into_a_shared_page_copies_it():
    c, m = pair()
    resize(c, m, [0], [64])
    write(c, m, 1, [0], [64], [0], 3)
    fork(c, m, [0, 0], [1, 2])
    resize(c, m, [1, 2], [40, 40])  # both end inside the page that slot 0 fills
    resize(c, m, [1], [41])
    write(c, m, 1, [1], [1], [40], 5)
    resize(c, m, [2, 0], [45, 65])
    resize(c, m, [0, 1, 2], [20, 20, 20])
    resize(c, m, [0, 1, 2], [30, 31, 32])  # two of the three hold the same page as each other still


def test_pages_run_out():
    c, m = pair(pages=7)
    resize(c, m, [0, 1, 2], [48, 64, 5])     # 3 + 4 pages; the third finds none
    resize(c, m, [2, 0, 3], [16, 0, 40])     # pages given up in the call serve its growing slots
    fork(c, m, [1, 3], [5, 6])               # nothing to copy for the first, no page for the second
    resize(c, m, [4, 5, 1], [200, 0, 0])     # past the table's width: skipped


def test_bad_entries_are_skipped():
    c, m = pair()
    resize(c, m, [0, 1, 0, 2], [20, 10, 99, 30])
    resize(c, m, [-1, 10, 3], [5, 5, 5])
    resize(c, m, [4, 5], [-1, 193])
    fork(c, m, [0, 1, 1, 11, 2], [7, 7, 0, 8, -2])
    k = tensor((3, 2, 32), 1, BF16, DEV)
    c.write(k, k, i32([0], DEV), i32([0, 3], DEV), i32([18], DEV))  # positions 18 .. 20 of a slot of 20
    st, detail = c.device_status()
    assert st == moe.MOE_ERR_DEVICE_CHECK and detail == 2
    m.write(0, [0], [0, 2], [18], k.cpu(), k.cpu())
    same(c, m)
    fork(c, m, [0], [9])
    c.write(k, k, i32([9], DEV), i32([0, 3], DEV), i32([2], DEV))  # a page that slot 0 holds too
    assert c.device_status()[0] == moe.MOE_ERR_DEVICE_CHECK
    same(c, m)


def test_compact():
    c, m = pair(pages=64, slots=12)
    resize(c, m, list(range(8)), [60, 100, 17, 33, 90, 1, 64, 130])
    write(c, m, 0, [1, 7], [100, 130], [0, 0], 2)
    fork(c, m, [1, 7], [8, 9])
    resize(c, m, [0, 2, 4], [0, 0, 0])
    compact(c, m)
    compact(c, m)  # nothing left to move
    resize(c, m, list(range(10)), [0] * 10)
    compact(c, m)


def test_copy_pages():
    c, m = pair()
    c.copy_pages(i32([3, 9, 5], DEV), i32([50, 0, 5], DEV))
    for a, b in ((3, 50), (9, 0)):
        m._copy(a, b)
    assert c.device_status() == (moe.MOE_OK, 0)
    same(c, m)
    c.copy_pages(i32([1, 60, 2], DEV), i32([40, 41, -1], DEV))
    assert c.device_status()[0] == moe.MOE_ERR_DEVICE_CHECK
    m._copy(1, 40)
    same(c, m)


def test_clear():
    c, m = pair()
    resize(c, m, [0, 4], [70, 20])
    c.clear()
    assert (c.table == -1).all() and (c.lens == 0).all() and (c.refs == 0).all()


@pytest.mark.parametrize("pages,slots,width", [(5000, 1500, 3), (9000, 40, 700), (70000, 64, 40), (24000, 100, 400)])
def test_large_tables(pages, slots, width):
    """More pages and slots than the table kernels handle in one step."""
    c, m = pair(layers=1, pages=pages, slots=slots, width=width, Hk=1, D=8)
    r = random.Random(pages)
    lens = [r.randint(0, width * 16) for _ in range(slots)]
    resize(c, m, list(range(slots)), lens)
    drop = r.sample(range(slots), slots // 2)
    resize(c, m, drop, [0] * len(drop))
    keep = [s for s in range(slots) if s not in set(drop)]
    half = len(drop) // 2
    fork(c, m, [r.choice(keep) for _ in range(half)], drop[:half])
    compact(c, m)
    resize(c, m, drop[half:], [r.randint(0, width * 16) for _ in drop[half:]])


@pytest.mark.parametrize("seed", range(12))
def test_random_histories(seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 64])
    c, m = pair(pages=r.choice([20, 60, 200]), page=page, slots=12, width=9, D=r.choice([8, 24, 64]),
                dtype=r.choice([BF16, F32]), seed=seed)
    for step in range(25):
        what = r.random()
        pick = r.sample(range(12), r.randint(1, 8))
        if what < 0.45:
            before = list(m.lens)
            resize(c, m, pick, [r.choice([0, m.lens[s], min(9 * page, m.lens[s] + r.randint(1, 2 * page)),
                                          r.randint(0, 9 * page)]) for s in pick])
            grown = [s for s in pick if m.lens[s] > before[s]]
            if grown:
                write(c, m, r.randrange(2), grown, [m.lens[s] - before[s] for s in grown], [before[s] for s in grown],
                      1000 * seed + step)
        elif what < 0.8:
            half = max(1, len(pick) // 2)
            fork(c, m, [r.choice(pick[:half]) for _ in pick[half:]], pick[half:]) if pick[half:] else None
        else:
            compact(c, m)


def test_cache_feeds_decode():
    """Slots grown, written, forked and compacted, then attended: the whole life of a small batch."""
    c, m = pair(pages=80, Hk=2, D=64, width=10)
    resize(c, m, [0], [70])
    write(c, m, 1, [0], [70], [0], 3)
    fork(c, m, [0] * 4, [1, 2, 3, 4])
    for step in range(12):
        slots = [0, 1, 2, 3, 4]
        before = [m.lens[s] for s in slots]
        resize(c, m, slots, [b + 1 + (s == 2) for s, b in zip(slots, before)])
        write(c, m, 1, slots, [1 + (s == 2) for s in slots], before, 50 + step)
        if step == 5:
            compact(c, m)
    q = tensor((5, 8, 64), 4, BF16, DEV)
    a = moe.Attention(8, 2, 64, BF16)
    for shared in (0, 64):
        lse = torch.empty((5, 8), device=DEV)
        out = a.decode(q, c, i32([0, 1, 2, 3, 4], DEV), layer=1, shared_len=shared, lse=lse)
        assert a.device_status() == (moe.MOE_OK, 0)
        for s in range(5):
            k, v = m.keys(1, s)
            check(out[s:s + 1], lse[s:s + 1], attend64(f64(q[s:s + 1]), k, v, [m.lens[s]], 0.125), m.lens[s], 64, BF16)


def test_calls_in_a_graph():
    c, m = pair()
    resize(c, m, [0, 1], [37, 5])
    slots, longer, shorter = i32([0, 1], DEV), i32([60, 25], DEV), i32([37, 5], DEV)
    k = tensor((43, 2, 32), 1, BF16, DEV)
    o = i32([0, 23, 43], DEV)
    with moe.GraphCapture(keep=(c, slots, longer, shorter, k, o)) as cap:
        c.resize(slots, shorter, stream=cap.stream)
        c.resize(slots, longer, stream=cap.stream)
        c.write(k, k, slots, o, shorter, layer=1, stream=cap.stream)
    for _ in range(3):
        cap.graph.launch()
    torch.cuda.synchronize()
    m.resize([0, 1], [60, 25])
    m.write(1, [0, 1], [0, 23, 43], [37, 5], k.cpu(), k.cpu())
    same(c, m)
