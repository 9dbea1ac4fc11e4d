// How attn_chunk.cu shares a chunk call out, on the host: its rules are the kernel's own (csrc/attn_plan.cuh), the threads
// and lanes that apply them are loops here.
#include <algorithm>
#include <vector>

#include "attn_plan.cuh"

using namespace moe;
using namespace moe::chunk;

namespace {
constexpr int kThreads = 384;

struct CtaPlan {
  long long all = 0, begin = 0, end = 0, x = 0;
  int run = 0, slot = 0, head = 0, runs = 0;
};
}  // namespace

// lens: positions of sequence i's slot as the plan reads them, found_lens: as the walk along the items does. An item found
// is 11 ints: CTA, kind, run, head, sequence, row0, rows, first block, block behind the last, all blocks, and the run that
// it ends in (-1: not begun here). Returns their number; -1: more steps than all heads' slots take; -2: more than `most`.
extern "C" int chunk_plan(const int32_t* qo, int n, int Tq, int G, int Hkv, int causal, const int32_t* lens,
                          const int32_t* found_lens, int ctas, int32_t* found, int most) {
  const int slots = (int)((long long)Tq * G / kRows + n);
  // the sequences in front of the first bad offsets
  int seqs = n;
  for (int i = n - 1; i >= 0; --i)
    if (bad_offsets(qo[i], qo[i + 1], Tq)) seqs = i;
  std::vector<int32_t> number(n);  // sequence i is in slot i
  for (int i = 0; i < n; ++i) number[i] = i;
  const int per = (slots + kThreads - 1) / kThreads;
  auto walk = [&](int thread, auto f) {
    const int s0 = std::min(slots, thread * per), s1 = std::min(slots, s0 + per);
    if (s0 < s1) walk_slots(qo, seqs, Tq, G, causal, s0, s1, [&](int i) { return lens[i]; }, f);
  };
  long long total[2] = {0, 0};
  std::vector<long long> sum(2 * kThreads, 0);
  for (int t = 0; t < kThreads; ++t)
    walk(t, [&](int, int kind, long long len) {
      sum[2 * t + kind] += len;
      total[kind] += len;
      return true;
    });
  int count = 0;
  for (int cta = 0; cta < ctas; ++cta) {
    CtaPlan plan[2];
    const Runs runs0(0, total[0] * Hkv, total[1] * Hkv, ctas);
    for (int kind = 0; kind < 2; ++kind) {
      CtaPlan& p = plan[kind];
      p.all = total[kind];
      p.run = run_of(kind, runs0, cta, ctas);
      if (p.all == 0) continue;
      const Runs runs(kind, total[0] * Hkv, total[1] * Hkv, ctas);
      p.runs = runs.n;
      if (p.run >= runs.n) continue;
      p.begin = runs.begin(p.run);
      p.end = runs.begin(p.run + 1);
      p.head = (int)(p.begin / p.all);
      const long long at = p.begin - p.head * p.all;
      long long x = 0;
      for (int t = 0; t < kThreads; x += sum[2 * t++ + kind]) {
        if (at < x || at >= x + sum[2 * t + kind]) continue;
        long long y = x;
        bool here = true;
        walk(t, [&](int s, int k, long long len) {
          if (k == kind && here) {
            p.slot = s;
            p.x = y - at;
            y += len;
            here = y <= at;
          }
          return here;
        });
      }
    }
    for (int kind = 0; kind < 2; ++kind) {
      const CtaPlan& p = plan[kind];
      if (p.begin == p.end) continue;
      Place at{p.x, p.slot & ~31, p.head};
      SlotItem ci[32];
      long long before[33];
      bool first = true;
      long long steps = 0;
      do {
        if (++steps > (long long)Hkv * (slots / 32 + 1)) return -1;
        before[0] = 0;
        for (int lane = 0; lane < 32; ++lane) {
          const int s = at.base + lane;
          ci[lane] = SlotItem{};
          if (s < slots)
            ci[lane] = slot_item(qo, number.data(), Tq, G, causal, s, find_tile_seq(qo, seqs, G, kRows, s),
                                 [&](int i) { return found_lens[i]; });
          if (item_kind(ci[lane].nrows) != kind) ci[lane].nrows = 0;
          before[lane + 1] = before[lane] + ci[lane].length();
        }
        if (first) at.x -= before[p.slot & 31];
        first = false;
        for (int lane = 0; lane < 32; ++lane) {
          const SlotItem& it = ci[lane];
          const int all = std::max(1, it.n_blocks);
          const int b0 = first_block(0, at.x + before[lane], all);
          const int b1 = first_block(p.end - p.begin, at.x + before[lane], all);
          if (it.nrows == 0 || b0 >= b1) continue;
          if (count == most) return -2;
          int end = -1;
          if (b0 == 0 && b1 < all)
            end = Runs(kind, total[0] * Hkv, total[1] * Hkv, ctas)
                      .of(p.begin + at.x + before[lane] + (long long)(all - 1) * kBlock);
          const int item[11] = {cta, kind, p.run, at.head, it.seq, it.row0, it.nrows, b0, b1, all, end};
          std::copy(item, item + 11, found + 11LL * count++);
        }
      } while (at.next(before[32], p.end - p.begin, slots, Hkv));
    }
  }
  return count;
}

// The tile kernels and their join: written[t] whether the tile of 64 rows of a slot has the first or the last row of token t,
// joined[t] whether the join, which looks for the token's own sequence (32 places a step, a lane each), takes those.
extern "C" void chunk_rows(const int32_t* qo, int n, int Tq, int G, uint8_t* written, uint8_t* joined) {
  constexpr int R = 64;
  const long long slots = (long long)Tq * G / R + n;
  auto ok = [&](int i) { return !bad_offsets(qo[i], qo[i + 1], Tq); };
  for (long long s = 0; s < slots; ++s) {
    const int i = find_tile_seq(qo, n, G, R, s);
    const long long r0 = (s - ((long long)qo[i] * G / R + i)) * R, rows = ok(i) ? (long long)(qo[i + 1] - qo[i]) * G : 0;
    for (long long r = r0; r0 >= 0 && r < std::min(rows, r0 + R); ++r)
      written[qo[i] + r / G] |= (r % G == 0 ? 1 : 0) | (r % G == G - 1 ? 2 : 0);
  }
  bool bad = false;
  for (int i = 0; i < n; ++i) bad = bad || !ok(i);
  for (int t = 0; t < Tq; ++t) {
    int i = 0, len = n;
    while (len > 1) {
      const int step = (len + 31) / 32;
      int k = -1;
      for (int lane = 0; lane < 32; ++lane) k += lane * step < len && qo[i + lane * step] <= t ? 1 : 0;
      const int skip = std::max(k, 0) * step;
      i += skip;
      len = std::min(len - skip, step);
    }
    if (!ok(i) || t < qo[i] || t >= qo[i + 1]) continue;
    for (int h = 0; h < G; h += std::max(1, G - 1)) {
      const long long slot = (long long)qo[i] * G / R + i + ((long long)(t - qo[i]) * G + h) / R;
      if (!bad || find_tile_seq(qo, n, G, R, slot) == i) joined[t] |= (h == 0 ? 1 : 0) | (h == G - 1 ? 2 : 0);
    }
  }
}
