// How packed rows are cut into tiles, and a chunk call's tiles shared out: arithmetic on offsets and lengths alone, which
// also compiles for the host.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_PLAN __device__ __forceinline__
#else
#define MOE_PLAN inline
#endif

namespace moe {

// A tile slot of packed prompts: with R rows a tile, sequence i (L_i tokens) owns the slots
// floor(q_offsets[i] G / R) + i up to the next sequence's first, which are never fewer than its
// ceil(L_i G / R) tiles. So tile slots are found from the offsets alone, with no scan over the
// sequences' tile counts: the largest i whose first slot is <= s, by bisection.
MOE_PLAN int find_tile_seq(const int32_t* qo, int n, int G, int R, long long s) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)qo[mid] * G / R + mid <= s) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Keys that query token t sees.
MOE_PLAN int visible_keys(int t, int nq, int nk, int causal) {
  if (!causal) return nk;
  const int lim = t + 1 + nk - nq;
  return lim < 0 ? 0 : (lim > nk ? nk : lim);
}

// Whether a sequence's offsets are out of order or range. Bisection needs them in order, and what looks for a sequence in two
// ways agrees only then: attn_chunk.cu's plan and its walk along the items take the sequences in front of the first one with
// such offsets, and the join behind the tile kernels asks whether a tile would have been found.
MOE_PLAN bool bad_offsets(int q0, int q1, int Tq) { return q0 < 0 || q1 < q0 || q1 > Tq; }

// ------------------------------------------------------------------ attn_chunk.cu
namespace chunk {

// How a chunk call is shared out. An item is, as for prompts, 256 packed rows of one key/value head. There are two kinds:
// those of two tiles (0) and those of one (1). The items of a kind lie in a row (heads outside, tile slots inside), each
// as long as its cost: kBlock a block of keys, and kItem for Q, the first scores and the results (measured with heads
// of 128, us: 1.45 a block and 6 of two tiles, 1.06 and 5.5 of one; heads of 64 are shared out by the same numbers). The
// row is cut into equally long runs, one a CTA, whatever items the cuts fall into; runs are not shorter than kShortest.
// A long call gives each CTA a run of either kind: the tensor cores bound the one and the memory the other, and CTAs
// that held more of one kind than others would end at another time than these. (8 chunks and 56 single tokens: 800 us
// with one row for both kinds, 690 so. Half of the CTAs begin with one kind and half with the other: 735 where all
// begin with the same.) That is one more cut item a CTA, so where all runs together are shorter than kBoth a CTA the
// kinds take CTAs of their own, in proportion to their times: 4 chunks of 2048 tokens together behind 8192, heads of 64,
// 125 us so and 141 with both kinds in each CTA; eight mixed batches of 220 us and more 422 so and 404 with both.
// A block belongs to the run that its beginning lies in. An item inside one run goes to the output; of one that
// several runs share, each puts its part (a piece) into the workspace, and chunk_join_kernel adds them up in order, so
// that results do not depend on which CTA is done first. A run has at most two such items, its first and its last: 2
// pieces a run are enough however long the keys.
constexpr int kTile = 128, kRows = 2 * kTile, kKeys = 128;  // rows of a tile and of an item, keys of a block
constexpr int kBlock = 4, kItem = 16, kShortest = 16, kBoth = 400;

template <typename T> MOE_PLAN T least(T a, T b) { return b < a ? b : a; }
template <typename T> MOE_PLAN T most(T a, T b) { return a < b ? b : a; }
MOE_PLAN int blocks_of(int keys) { return (keys + kKeys - 1) / kKeys; }
MOE_PLAN int item_kind(int rows) { return rows <= kTile ? 1 : 0; }
// Length of an item of so many blocks.
MOE_PLAN long long item_length(int blocks) { return kItem + (long long)blocks * kBlock; }

// What fills a tile slot (nrows = 0: nothing).
struct SlotItem {
  int seq, row0, nrows, q0, nq, nk, slot;
  int lim0, lim1, n_blocks;  // keys that the tiles' last rows see; blocks of keys
  MOE_PLAN long long length() const { return nrows > 0 ? item_length(n_blocks) : 0; }
};
// Of tile slot s, where sequence i is the one that may fill it. slot: the sequence's in the cache, len(slot) the positions
// that it holds.
template <typename Len>
MOE_PLAN SlotItem slot_item(const int32_t* qo, const int32_t* slots, int Tq, int G, int causal, int s, int i, Len len) {
  SlotItem it{};
  it.seq = i;
  const int q0 = qo[i], q1 = qo[i + 1];
  it.slot = slots[i];
  if (bad_offsets(q0, q1, Tq)) return it;
  it.q0 = q0;
  it.nq = q1 - q0;
  const long long r0 = ((long long)s - ((long long)q0 * G / kRows + i)) * kRows;
  if (r0 < 0 || r0 >= (long long)it.nq * G) return it;
  it.nk = len(it.slot);
  it.row0 = (int)r0;
  it.nrows = least(kRows, it.nq * G - it.row0);
  it.lim0 = visible_keys((it.row0 + least(it.nrows, kTile) - 1) / G, it.nq, it.nk, causal);
  it.lim1 = it.nrows > kTile ? visible_keys((it.row0 + it.nrows - 1) / G, it.nq, it.nk, causal) : 0;
  it.n_blocks = blocks_of(most(it.lim0, it.lim1));
  return it;
}

// f(slot, kind, length) for the slots of [s0, s1) that an item fills, as long as it returns true. The sequences lie in the
// slots' order, so what is read of them (len(i): the positions of sequence i) is read ahead, four at a time.
template <typename Len, typename F>
MOE_PLAN void walk_slots(const int32_t* qo, int n, int Tq, int G, int causal, int s0, int s1, Len len, F f) {
  int s = s0, i = find_tile_seq(qo, n, G, kRows, s0);
  while (s < s1 && i < n) {
    int q[5], held[4];
#pragma unroll
    for (int k = 0; k < 5; ++k) q[k] = qo[least(i + k, n)];
#pragma unroll
    for (int k = 0; k < 4; ++k) held[k] = len(least(i + k, n - 1));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k >= n || bad_offsets(q[k], q[k + 1], Tq)) continue;
      const long long first = (long long)q[k] * G / kRows + i + k, rows = (long long)(q[k + 1] - q[k]) * G;
      const long long end = least((long long)s1, first + (rows + kRows - 1) / kRows);
      for (s = most(s, (int)least(first, (long long)s1)); s < end; ++s) {
        const int row0 = (int)(s - first) * kRows, nrows = least(kRows, (int)rows - row0), nq = q[k + 1] - q[k];
        const int lim0 = visible_keys((row0 + least(nrows, kTile) - 1) / G, nq, held[k], causal);
        const int lim1 = nrows > kTile ? visible_keys((row0 + nrows - 1) / G, nq, held[k], causal) : 0;
        if (!f(s, item_kind(nrows), item_length(blocks_of(most(lim0, lim1))))) return;
      }
    }
    i += 4;
  }
}

// The runs of a kind: how many, their beginnings, and the run that place x lies in. t0, t1: the lengths of the two rows.
struct Runs {
  long long all;
  int n;
  MOE_PLAN Runs(int kind, long long t0, long long t1, int ctas) : all(kind ? t1 : t0) {
    long long runs = ctas;
    // (a block of one tile takes 3/4 as long)
    if (t0 > 0 && t1 > 0 && ctas > 1 && 4 * t0 + 3 * t1 < 4LL * kBoth * ctas) {
      const long long ones = least(ctas - 1LL, ctas * (3 * t1) / (4 * t0 + 3 * t1) + 1);
      runs = kind ? ones : ctas - ones;
    }
    n = (int)most(1LL, least(runs, all / kShortest));
  }
  MOE_PLAN long long begin(int c) const { return all * c / n; }
  MOE_PLAN int of(long long x) const {  // (the last one behind the end: pieces are numbered by it)
    const int c = (int)(((x + 1) * n - 1) / all);
    return least(c, n - 1);
  }
};
// Which run of a kind a CTA takes: those of kind 1 go on where those of kind 0 end, so that a short call's lie in CTAs of
// their own.
MOE_PLAN int run_of(int kind, const Runs& runs0, int cta, int ctas) {
  if (kind == 0) return cta;
  const int c = cta - (runs0.all > 0 ? runs0.n % ctas : 0);
  return c < 0 ? c + ctas : c;
}

// Where a walk along a run's items is: 32 slots from `base` on of a head, whose first item's place is x from the run's
// beginning on.
struct Place {
  long long x;
  int base, head;
  // Goes on to the next slots, behind a batch whose items are so long together. False behind the run's end, and behind the
  // last head whatever the lengths are: nothing that is read on the way makes the walk longer.
  MOE_PLAN bool next(long long length, long long run, int slots, int heads) {
    x += length;
    base += 32;
    if (base >= slots) {
      base = 0;
      ++head;
    }
    return x < run && head < heads;
  }
};
// The first block of an item of `blocks` ones at place `at` that does not begin in front of p.
MOE_PLAN int first_block(long long p, long long at, int blocks) {
  p -= at;
  return p <= 0 ? 0 : (int)least((long long)blocks, (p + kBlock - 1) / kBlock);
}

}  // namespace chunk
}  // namespace moe
