"""How a chunk call over the cache is shared out among CTAs (csrc/attn_plan.cuh), compiled for the host: every block of every
item once, pieces where the join looks for them, and ends and bounds whatever the offsets and lengths hold."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_moe_gb300", "csrc")
TILE, ROWS, KEYS = 128, 256, 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, os.path.join(ROOT, "tests", "chunk_plan.cpp"),
                    "-o", path], check=True)
    return ctypes.CDLL(path)


@pytest.fixture(scope="module")
def plan(lib):
    f = lib.chunk_plan

    def run(offs, Tq, G, Hkv, lens, found_lens=None, causal=True, ctas=152):
        """The items found: tuples (CTA, kind, run, head, sequence, row0, rows, b0, b1, blocks, last run)."""
        n = len(lens)
        assert len(offs) == n + 1
        out = np.zeros((20000, 11), dtype=np.int32)
        arrays = [np.ascontiguousarray(x, dtype=np.int32) for x in (offs, lens, lens if found_lens is None else found_lens)]
        at = [a.ctypes.data_as(ctypes.c_void_p) for a in arrays]
        got = f(at[0], n, Tq, G, Hkv, int(causal), at[1], at[2], ctas, out.ctypes.data_as(ctypes.c_void_p), len(out))
        assert got >= 0, "steps without end" if got == -1 else "more items than room"
        return [tuple(x) for x in out[:got].tolist()]
    return run


def good(offs, Tq):
    """The sequences in front of the first one whose offsets are out of order or range."""
    for i, (a, b) in enumerate(zip(offs, offs[1:])):
        if a < 0 or b < a or b > Tq:
            return i
    return len(offs) - 1


def visible(t, nq, nk, causal):
    return min(nk, max(0, t + 1 + nk - nq)) if causal else nk


def expected(offs, Tq, G, Hkv, lens, causal):
    """{(head, sequence, row0): (rows, blocks)} of a call."""
    want = {}
    for i in range(good(offs, Tq)):
        nq = offs[i + 1] - offs[i]
        for r in range(0, nq * G, ROWS):
            rows = min(ROWS, nq * G - r)
            ends = {r + min(rows, TILE) - 1, r + rows - 1}
            keys = max(visible(e // G, nq, lens[i], causal) for e in ends)
            for h in range(Hkv):
                want[h, i, r] = rows, max(1, -(-keys // KEYS))
    return want


def check(items, offs, Tq, G, Hkv, lens, causal=True):
    want, blocks = expected(offs, Tq, G, Hkv, lens, causal), {}
    pieces = {}  # (kind, run): of the items that began in an earlier one, at most one
    for cta, kind, run, h, seq, r, rows, b0, b1, n, end in items:
        assert want[h, seq, r] == (rows, n) and kind == (rows <= TILE)
        blocks.setdefault((h, seq, r), []).append((b0, b1, run, end))
        if b0 > 0:
            assert (kind, run) not in pieces
            pieces[kind, run] = h, seq, r
    assert blocks.keys() == want.keys()
    cut = set()
    for key, parts in blocks.items():
        parts.sort()
        assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == want[key][1]
        kind, first, end = int(want[key][0] <= TILE), parts[0][2], parts[0][3]
        # a cut item lies in the runs from its first one to `end`, which is where its pieces are added up from
        assert [p[2] for p in parts] == list(range(first, first + len(parts)))
        assert end == (first + len(parts) - 1 if len(parts) > 1 else -1)
        if len(parts) > 1:
            assert (kind, first) not in cut
            cut.add((kind, first))


def draw(r):
    n, G, Hkv = r.randint(1, 9), r.choice([1, 2, 4, 7, 8]), r.choice([1, 2, 5])
    nq = [r.choice([0, 1, 2, 5, r.randint(1, 40), r.randint(1, 700)]) for _ in range(n)]
    lens = [r.choice([0, a, a + r.randint(0, 300), r.randint(0, 5000)]) for a in nq]
    offs = [sum(nq[:i]) for i in range(n + 1)]
    return offs, offs[-1] + r.choice([0, 0, 3]), G, Hkv, lens, r.choice([True, True, False]), r.choice([152, 148, 37, 5, 1])


@pytest.mark.parametrize("seed", range(40))
def test_every_block_once(plan, seed):
    r = random.Random(seed)
    for _ in range(6):
        offs, Tq, G, Hkv, lens, causal, ctas = draw(r)
        check(plan(offs, Tq, G, Hkv, lens, causal=causal, ctas=ctas), offs, Tq, G, Hkv, lens, causal)


def test_many_sequences(plan):
    r = random.Random(1)
    nq = [r.choice([0, 1, 1, 3, 200]) for _ in range(900)]
    offs = [sum(nq[:i]) for i in range(901)]
    lens = [a + r.randint(0, 300) for a in nq]
    check(plan(offs, offs[-1], 4, 2, lens), offs, offs[-1], 4, 2, lens)


# Sequences behind bad offsets that a bisection over all of them misses and a walk from the first finds.
@pytest.mark.parametrize("offs,Tq,G,Hkv,lens", [
    ([0, 1000, 200, 600], 600, 4, 2, [900] * 3),
    ([0, 68, 71, 195, 103, 128, 300], 300, 4, 2, [436, 2752, 56, 2755, 2210, 2195]),
    ([0, 971, 1679, 1080, 1145], 1679, 1, 1, [2500] * 4),
    ([0, 4, 99, 15], 15, 2, 2, [100, 200, 60]),
    ([0, 300, 200, 500], 500, 2, 2, [400, 400, 400]),
    ([5, 3, 10], 10, 2, 2, [50, 50]),
    ([-1, 3, 10], 10, 2, 2, [50, 50]),
    ([0, 3, 2 ** 31 - 1, 10], 10, 8, 2, [50, 50, 50]),
    ([0, 3, -2 ** 31, 10], 10, 8, 2, [50, 50, 50]),
])
def test_sequences_end_in_front_of_bad_offsets(plan, offs, Tq, G, Hkv, lens):
    for ctas in (152, 8, 1):
        check(plan(offs, Tq, G, Hkv, lens, ctas=ctas), offs, Tq, G, Hkv, lens)


@pytest.mark.parametrize("kind", ["decreasing", "any", "many"])
@pytest.mark.parametrize("seed", range(30))
def test_random_bad_offsets(plan, seed, kind):
    r = random.Random(seed)
    for _ in range(8):
        offs, Tq, G, Hkv, lens, causal, ctas = draw(r)
        for _ in range(4 if kind == "many" else 1):
            i = r.randrange(len(offs))
            offs[i] = r.randint(0, max(1, Tq)) if kind == "decreasing" else r.choice(
                [-1, Tq + 1, 2 * Tq + 5, 2 ** 31 - 1, -2 ** 31, r.randint(-50, Tq + 50)])
        check(plan(offs, Tq, G, Hkv, lens, causal=causal, ctas=ctas), offs, Tq, G, Hkv, lens, causal)


@pytest.mark.parametrize("seed", range(30))
def test_joined_rows_are_written(lib, seed):
    """The tile kernels find a slot's sequence, their join a token's. It takes no row that no tile wrote, and over good offsets
    every sequence's."""
    r = random.Random(seed)
    for k in range(16):
        offs, Tq, G, _, lens, _, _ = draw(r)
        if k % 4 == 0:  # more sequences than the join's lanes
            nq = [r.choice([0, 1, 3]) for _ in range(r.randint(33, 200))]
            offs, Tq, lens = [sum(nq[:i]) for i in range(len(nq) + 1)], sum(nq), nq
        for _ in range(k % 3):
            offs[r.randrange(len(offs))] = r.choice([r.randint(0, Tq), r.randint(-50, Tq + 50), 2 ** 31 - 1, -2 ** 31])
        at = np.array(offs, dtype=np.int32)
        written, joined = np.zeros(Tq + 1, dtype=np.uint8), np.zeros(Tq + 1, dtype=np.uint8)
        lib.chunk_rows(at.ctypes.data_as(ctypes.c_void_p), len(lens), Tq, G, written.ctypes.data_as(ctypes.c_void_p),
                       joined.ctypes.data_as(ctypes.c_void_p))
        assert (joined & ~written == 0).all()
        if good(offs, Tq) == len(lens):
            assert (joined[offs[0]:offs[-1]] == 3).all() and not joined[offs[-1]:].any() and (joined == written).all()


@pytest.mark.parametrize("seed", range(30))
def test_lengths_that_change_on_the_way_stay_in_bounds(plan, seed):
    """Lengths read again are others: the results are anyone's, but the walk ends, and heads, runs and rows exist."""
    r = random.Random(seed)
    for _ in range(8):
        offs, Tq, G, Hkv, lens, causal, ctas = draw(r)
        other = [r.choice([0, x, 5000, r.randint(0, 9000)]) for x in lens]
        for _, kind, run, h, seq, row0, rows, b0, b1, n, end in plan(offs, Tq, G, Hkv, lens, other, causal, ctas):
            nq = offs[seq + 1] - offs[seq]
            assert 0 <= h < Hkv and 0 <= run < ctas and 0 <= row0 and row0 + rows <= nq * G and 0 <= b0 < b1 <= n
            assert end == -1 or run <= end < ctas
